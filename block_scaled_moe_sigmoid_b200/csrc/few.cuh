// Matrix products with MXFP4 weights for a few token rows (T <= 16): a stream of the weights.
//
//   FEW_LINEAR  y[t] = W x[t]                                    one matrix, x in MXFP8
//   FEW_GLU     h[t,e] = MX(glu(Wg x[t], Wu x[t]))               the experts e = idx[t][j]
//               v[t] = bf16(glu(Vg x[t], Vu x[t]))               the shared expert, bf16
//   FEW_DOWN    y[t] = bf16(Vd v[t] + sum_j w[t][j] Wd h[t,j])   the same experts
//
// With so few rows every weight byte is used once and the bytes are the cost: 17/32 byte per
// weight at the copy rate of the memory.  The work is one list of steps, a step being one 256-row
// x 128-column tile of packed weights (16 KB of codes, one contiguous block, and 1 KB of scales).
// CTA c of G takes the steps [c S / G, (c + 1) S / G): every SM streams the same number of bytes
// whatever the number of experts, rows or columns.  (The grouped GEMM gives a CTA whole tiles: one
// token's 16 experts make 384 of them, 2.6 per SM.)  Where a CTA's range begins or ends inside a
// tile's contraction it writes an fp32 partial, and the CTA that arrives last at the tile's counter
// adds the partials in the order of the CTAs (a fixed order: results do not depend on timing) and
// finishes the tile.  No CTA waits for another.
//
// FEW_DOWN contracts over (expert, column) in one go: a tile of y takes the experts one after the
// other, each through an accumulator of its own that the epilogue adds, times the token's weight, to
// fp32 registers.
//
// The shared expert's bf16 weights are steps of the same lists: 256 rows x 64 columns, 32 KB, counted
// as two (a boundary between two CTAs that falls inside one gives it to the first).  In FEW_GLU they
// are tiles of their own after the routed ones, in FEW_DOWN they end each tile's contraction.  Their
// MMAs are kind::f16; everything else is common.
//
// A step's products are eight tcgen05.mma kind::mxf8f6f4.block_scale (two 128-row halves x four
// 32-column blocks, N = 16 tokens), which decode the codes and apply the scales themselves.  The same
// products on mma.sync were measured too: making f16 operands out of the codes then takes more than
// the load (40000 x 7168, 8 rows: cvt 3.0 TB/s, half of it by bit moves 2.6 TB/s, E4M3 operands 2.4 TB/s).
//
// Roles (416 threads): warp 0 loads weight tiles and their scales, warp 10 the token rows (a 16-row
// box per step), warp 11 moves each step's scales into TMEM, warps 1 and 12 issue the MMAs of one
// 128-row half each (one thread forms and issues an instruction in about 90 cycles, and eight of them
// would take longer than the step's load), warps 2 to 9 run the epilogue, a thread per weight row.
// The scale and MMA warps run converged and elect the lane that issues: formed in a branch of one lane,
// each operand goes to its uniform register by itself, and the scale warp alone then held the stream at
// 5.9 TB/s.
//
// Measured (B200, copy rate 6.54 TB/s; replayed on one set of weights): 8 tokens on 57 experts of 3584 x 3072
// in 150 us, 6.7 TB/s; one token on 16 experts of 7168 x 3072 in 91.0 us, 6.2 TB/s (112 us with a shared
// expert, 115 over three sets of weights); 8 rows of 40000 x 7168 in 26.9 us, 5.7 TB/s.  Around the stream
// each kernel takes about 4 us for its tables, the first load's latency and the last exchange; small shapes
// are that latency.
#pragma once
#include <type_traits>

#include "gemm.cuh"
#include "kernels.cuh"

namespace moe {

enum { FEW_LINEAR = 0, FEW_GLU = 1, FEW_DOWN = 2 };
constexpr int kFewRows = 16;                   // tokens per call: the MMA's N
constexpr int kFewThreads = 416;
constexpr int kFewTile = 256 * 64;             // bytes of codes per step
constexpr int kFewATile = 256 * 128;           // the same in shared memory, a byte per code
constexpr int kFewBTile = kFewRows * 128;
constexpr int kFewStage = kFewATile + kFewBTile;
constexpr int kFewSF = 1024 + 512;             // weight and token scale atoms per stage
constexpr int kFewMaxStages = 6;
constexpr int kFewPart = kFewRows * 256;       // floats of a partial
constexpr int kFewMaxCtas = 256;               // bound on the grid (sizes partials and counters)
constexpr int kFewSmemMax = 232448;
constexpr int kFewTmemCols = 256;              // two accumulators of 2 x 16 columns, 16 columns of scales per stage
static_assert(kFewStage % 1024 == 0, "swizzled tiles start on 1024 bytes");
static_assert(64 + 16 * kFewMaxStages <= kFewTmemCols, "TMEM budget");

// Division of 0 <= n < 2^31 by a d known on the host: n * ceil(2^(31 + s) / d) >> (31 + s), s = ceil(log2 d).
// The roles divide before their first step, and an integer division is a call's worth of instructions to
// fetch and run: with the host's factors 1 x 7168 x 7168 takes 10.1 us against 10.5.
struct FastDiv {
  int d;
  uint32_t mul;
  int shift;
  __device__ __forceinline__ int div(int n) const { return d == 1 ? n : (int)(__umulhi((uint32_t)n, mul) >> shift); }
};
inline FastDiv fast_div(int d) {
  int s = 0;
  while ((1ll << s) < d) ++s;
  const uint32_t mul = d == 1 ? 0u : (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
  return {d, mul, s - 1};
}

struct FewArgs {
  int T, k, E;
  int m_tiles, k_tiles;   // of one matrix
  FastDiv by_m, by_k;     // by m_tiles, k_tiles,
  FastDiv by_ss;          // the units of a tile's shared part,
  FastDiv by_grid;        // and the number of CTAs
  int rows;               // valid output rows (FEW_LINEAR, FEW_DOWN)
  int stages;
  const uint8_t* sf;      // weight scales, [matrix][m-tile][k-tile][1 KB]
  const int* idx;
  const float* w;
  const uint8_t* xs;      // FEW_LINEAR, FEW_GLU: token scales [T][4 k_tiles]
  int sh_tiles, sh_steps; // shared expert: m-tiles (FEW_GLU), 64-column steps of a tile's contraction (0: none)
  __nv_bfloat16* hsh;     // FEW_GLU: its hidden values [T][128 sh_tiles]
  uint8_t* hq;            // codes of h, [used expert][T][128 k-tiles of the down product]
  uint8_t* hs;            // scale atoms of h, [used expert][k-tile][512]
  void* y;
  int y_f32;
  float* part;            // [2 per CTA][16][256]
  unsigned int* counters; // [CTAs], zero between launches
  unsigned int* status;
};

// Shared-memory layout (byte offsets from a 1024-byte aligned base); host and device agree on it.
struct FewSmem {
  int sf, ctrl, xs, red, tab, total;
};
__host__ __device__ inline FewSmem few_smem(int mode, int T, int k, int k_tiles, int stages) {
  FewSmem s;
  int o = stages * kFewStage;
  s.sf = o; o += stages * kFewSF;
  s.ctrl = o; o += 512;
  s.xs = o; if (mode != FEW_DOWN) o += T * k_tiles * 4;              // token scales
  s.red = o; if (mode == FEW_GLU) o += T * 128 * 4;                  // up values on their way to the gates
  s.tab = o; if (mode != FEW_LINEAR) o += (256 + 4 * T * k) * 4;     // experts in use
  if (mode == FEW_DOWN) o += T * k * T * 4;                          // and their tokens' weights
  s.total = o + 1024;
  return s;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ unsigned int count_acq_rel(unsigned int* counter) {
  unsigned int v;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(v) : "l"(counter) : "memory");
  return v;
}
// Order this thread's shared-memory writes before later asynchronous-proxy reads (tcgen05.cp).
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Steps that stay together in a CTA: a whole tile, or one step.  Split tiles cost the exchange of
// partials, about 3 us at the end of the call, the time of kFewSplitCost steps; whole tiles cost the
// last wave's idle CTAs (5 rows of 1003 x 640, four tiles of five steps: 5.8 us whole, 8.0 split).
constexpr int kFewSplitCost = 8;
__device__ __forceinline__ int few_unit(int tiles, int KT, const FastDiv& by_grid) {
  const int up = by_grid.d - 1;
  return by_grid.div(tiles + up) * KT <= by_grid.div(tiles * KT + up) + kFewSplitCost ? KT : 1;
}
__device__ __forceinline__ bool elect_one() {   // one lane of the converged warp, the same one each time
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void few_bar() {   // the epilogue warps
  asm volatile("bar.sync 1, 256;" ::: "memory");
}

template <int MODE, int ACT>
__global__ void __launch_bounds__(kFewThreads, 1)
    few_kernel(const __grid_constant__ FewArgs a, const __grid_constant__ CUtensorMap tmW,
               const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmSW,
               const __grid_constant__ CUtensorMap tmSX) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const FewSmem L = few_smem(MODE, a.T, a.k, a.k_tiles, a.stages);
  uint64_t* full_bar = (uint64_t*)(smem + L.ctrl);
  uint64_t* empty_bar = full_bar + kFewMaxStages;
  uint64_t* sf_full = empty_bar + kFewMaxStages;
  uint64_t* acc_full = sf_full + kFewMaxStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;             // [2]
  uint64_t* drain_bar = acc_empty + 2;
  uint64_t* drain_sf = drain_bar + 1;
  uint32_t* tmem_holder = (uint32_t*)(drain_sf + 1);
  volatile int* abort_flag = (volatile int*)(tmem_holder + 1);
  int* fills = (int*)(tmem_holder + 2);           // [5]: weight producer, token producer, scale warp, MMA halves
  volatile int* s_last = fills + 5;
  int* s_used = fills + 6;
  // experts in use
  const int slots = a.T * a.k;
  uint32_t* bitmap = (uint32_t*)(smem + L.tab);
  int* prefix = (int*)(bitmap + 128);             // used experts before each word
  int* elist = prefix + 128;                      // the used experts, ascending
  int* tokens = elist + slots;                    // [used expert]: a bit for each token that uses it
  int* s_idx = tokens + slots;
  float* s_w = (float*)(s_idx + slots);
  float* hw = s_w + slots;                        // [used expert][T]: the token's routing weight

  // values that the compiler cannot see are the same in a warp come through a shuffle: what depends on
  // them then lives in uniform registers, where the MMA operands have to be
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(smem_u32(full_bar + s), 3);                          // two producers, the scale warp's commit
      mbar_init(smem_u32(empty_bar + s), 2);                         // both issuers
      mbar_init(smem_u32(sf_full + s), MODE == FEW_DOWN ? 2 : 1);    // weight scales, and h's
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(acc_full + b), 2);
      mbar_init(smem_u32(acc_empty + b), 8);
    }
    mbar_init(smem_u32(drain_bar), 2);
    mbar_init(smem_u32(drain_sf), 1);
    *abort_flag = 0;
    for (int r = 0; r < 5; ++r) fills[r] = 0;
    fence_mbar_init();
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
    if (MODE != FEW_LINEAR && a.sh_steps) {
      prefetch_tmap(&tmSW);
      prefetch_tmap(&tmSX);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), kFewTmemCols);
    tmem_relinquish();
  }
  // FEW_DOWN always follows FEW_GLU, which lets it start only after its own wait: all that was
  // launched before FEW_GLU is done by then, the ids, the routing weights and the packed weights
  // among it.  So its tables and weight loads begin here, and what FEW_GLU writes, and every buffer
  // that it shares with it, waits (token producer, epilogue).
  if (MODE != FEW_DOWN) griddep_wait();
  griddep_launch_dependents();
  // loads that the first barrier covers: the ids, or the token scales
  if constexpr (MODE != FEW_LINEAR) {
    for (int i = tid; i < slots; i += kFewThreads) {
      s_idx[i] = __ldcg(a.idx + i);   // past L1: FEW_DOWN reads before its wait
      tokens[i] = 0;
    }
    for (int i = tid; i < 128; i += kFewThreads) bitmap[i] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_holder, 0);

  int used = 1;
  if constexpr (MODE != FEW_LINEAR) {
    for (int i = tid; i < slots; i += kFewThreads) {
      const int e = s_idx[i];
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
    used = __shfl_sync(0xffffffffu, *s_used, 0);
    for (int i = tid; i < slots; i += kFewThreads) {
      const int e = s_idx[i];
      if (e < 0 || e >= a.E) continue;
      const int u = prefix[e >> 5] + __popc(bitmap[e >> 5] & ((1u << (e & 31)) - 1u));
      elist[u] = e;
      atomicOr(&tokens[u], 1 << (i / a.k));
    }
    __syncthreads();
  }

  // The list of steps, and this CTA's part [s0, s1) of it, in units of one routed step.
  const int SS = MODE == FEW_LINEAR ? 0 : 2 * a.sh_steps;                    // of a tile's shared part
  const int RT = MODE == FEW_DOWN ? used * a.k_tiles : a.k_tiles;            // of a tile's routed part
  const int KT = MODE == FEW_DOWN ? RT + SS : RT;                            // of a tile (FEW_GLU: a routed one)
  const int routed = MODE == FEW_GLU ? used * a.m_tiles * RT : a.m_tiles * KT;
  const int total = routed + (MODE == FEW_GLU ? a.sh_tiles * SS : 0);
  const int all_tiles = MODE == FEW_GLU ? used * a.m_tiles : a.m_tiles;
  const int unit = SS ? 1 : few_unit(all_tiles, KT, a.by_grid);              // steps that stay together
  const bool whole_tiles = unit == KT && !SS;
  const int units = whole_tiles ? all_tiles : total;
  // at least four steps for a CTA where tiles are split; the first `rem` CTAs take one unit more
  const int G = min(whole_tiles ? units : max(units >> 2, min(units, 1)), a.by_grid.d);
  const int c = blockIdx.x, per = G == a.by_grid.d ? a.by_grid.div(units) : units / max(G, 1), rem = units - per * G;
  const int s0 = c < G ? (c * per + min(c, rem)) * unit : 0, s1 = c < G ? s0 + (per + (c < rem)) * unit : 0;
  // the CTA with step s (unit = 1)
  auto cta_of = [&](int s) { return s < rem * (per + 1) ? s / (per + 1) : rem + (s - rem * (per + 1)) / per; };
  // A run: consecutive steps of one matrix and one tile, accumulated in TMEM: K tiles [kb, kb + n).
  // The tile is [t0, t0 + len) in the list, and its last step begins at t0 + last.
  struct Run { int tile, u, m, kb, n, next, t0, len, last; bool shared; };
  auto run_at = [&](int s) {
    Run r;
    r.u = 0;
    r.shared = false;
    int kk;   // place in the tile
    if (MODE == FEW_GLU && s >= routed) {
      r.shared = true;
      r.len = SS;
      r.tile = a.by_ss.div(s - routed);
      r.t0 = routed + r.tile * SS;
      r.m = r.tile;
      kk = s - r.t0;
    } else {
      r.len = KT;
      r.tile = MODE == FEW_DOWN ? s / KT : a.by_k.div(s);
      r.t0 = r.tile * KT;
      r.m = r.tile;
      kk = s - r.t0;
      if (MODE == FEW_GLU) {
        r.u = a.by_m.div(r.tile);
        r.m = r.tile - r.u * a.m_tiles;
      } else if (MODE == FEW_DOWN) {
        r.shared = kk >= RT;
        if (r.shared) kk -= RT;
        else r.u = a.by_k.div(kk), kk -= r.u * a.k_tiles;
      }
    }
    const int room = min(r.shared ? SS - kk : a.k_tiles - kk, s1 - s);
    r.kb = r.shared ? (kk + 1) >> 1 : kk;
    r.n = r.shared ? ((kk + room + 1) >> 1) - r.kb : room;   // 0: the second half of a step
    r.next = s + room;
    r.last = r.len - ((MODE == FEW_GLU ? r.shared : SS > 0) ? 2 : 1);
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
        const int e = MODE == FEW_LINEAR || r.shared ? 0 : elist[r.u];
        const size_t blk = ((size_t)e * a.m_tiles + r.m) * a.k_tiles + r.kb;
        auto run_steps = [&](auto shared) {
          for (int i = 0; i < r.n; ++i) {
            ok = mbar_wait(smem_u32(empty_bar + stage), phase ^ 1, a.status, abort_flag);
            if (!ok) return;
            const uint32_t sb = smem_u32(sf_full + stage), fb = smem_u32(full_bar + stage), dst = smem_u32(smem + stage * kFewStage);
            if constexpr (decltype(shared)::value) {
              mbar_arrive(sb);
              mbar_arrive_expect_tx(fb, kFewATile);
              tma_load_2d(dst, &tmSW, fb, (r.kb + i) * 64, r.m * 256, pol);
            } else {
              mbar_arrive_expect_tx(sb, 1024);
              bulk_load(smem_u32(smem + L.sf + stage * kFewSF), a.sf + (blk + i) * 1024, 1024, sb);
              mbar_arrive_expect_tx(fb, kFewTile);
              tma_load_2d(dst, &tmW, fb, 0, (int)((blk + i) * 256), pol);
            }
            ++nfill;
            if (++stage == a.stages) { stage = 0; phase ^= 1; }
          }
        };
        if (MODE != FEW_LINEAR && r.shared) run_steps(std::true_type{});
        else run_steps(std::false_type{});
        s = r.next;
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
      if (MODE == FEW_DOWN) griddep_wait();
      for (int s = s0; s < s1 && ok;) {
        const Run r = run_at(s);
        for (int i = 0; i < r.n; ++i) {
          ok = mbar_wait(smem_u32(empty_bar + stage), phase ^ 1, a.status, abort_flag);
          if (!ok) break;
          const uint32_t fb = smem_u32(full_bar + stage);
          if (MODE != FEW_LINEAR && r.shared) {
            if (MODE == FEW_DOWN) mbar_arrive(smem_u32(sf_full + stage));
            mbar_arrive_expect_tx(fb, kFewBTile);
            tma_load_2d(smem_u32(smem + stage * kFewStage + kFewATile), &tmSX, fb, (r.kb + i) * 64, 0, pol);
            ++nfill;
            if (++stage == a.stages) { stage = 0; phase ^= 1; }
            continue;
          }
          if constexpr (MODE == FEW_DOWN) {
            const uint32_t sb = smem_u32(sf_full + stage);
            mbar_arrive_expect_tx(sb, 512);
            bulk_load(smem_u32(smem + L.sf + stage * kFewSF + 1024), a.hs + ((size_t)r.u * a.k_tiles + r.kb + i) * 512, 512, sb);
          }
          mbar_arrive_expect_tx(fb, kFewBTile);
          // rows past the operand's tokens are another expert's, or zeros behind the tensor's end:
          // they reach accumulator columns that nothing reads
          tma_load_2d(smem_u32(smem + stage * kFewStage + kFewATile), &tmX, fb, (r.kb + i) * 128,
                      MODE == FEW_DOWN ? r.u * a.T : 0, pol);
          ++nfill;
          if (++stage == a.stages) { stage = 0; phase ^= 1; }
        }
        s = r.next;
      }
      fills[1] = nfill;
    }
    __syncwarp();
  } else if (warp == 11) {
    // ------------------------------------------------------------- scale factors -> TMEM
    const uint32_t* xs = (const uint32_t*)(smem + L.xs);
    if (MODE != FEW_DOWN) asm volatile("bar.sync 2, 288;" ::: "memory");   // the epilogue warps have loaded xs
    const uint64_t sf_desc0 = smem_desc(smem_u32(smem + L.sf), 16, 128, 0);
    int stage = 0, nfill = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int s = s0; s < s1 && ok;) {
      const Run r = run_at(s);
      if (MODE != FEW_LINEAR && r.shared) {   // no scales
        for (int i = 0; i < r.n; ++i) {
          int got = 1;
          if (lane == 0) got = mbar_wait(smem_u32(sf_full + stage), phase, a.status, abort_flag);
          ok = __shfl_sync(0xffffffffu, got, 0) != 0;
          if (!ok) break;
          if (lane == 0) mbar_arrive(smem_u32(full_bar + stage));
          ++nfill;
          if (++stage == a.stages) { stage = 0; phase ^= 1; }
        }
        s = r.next;
        continue;
      }
      for (int i = 0; i < r.n; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(sf_full + stage), phase, a.status, abort_flag));
        if (!ok) break;
        if constexpr (MODE != FEW_DOWN) {
          // the token scales' atom: row t's four bytes at 16 t (its last reader, the copy of the
          // stage's previous round, finished before the stage was released)
          if (lane < kFewRows)
            *(uint32_t*)(smem + L.sf + stage * kFewSF + 1024 + 16 * lane) = lane < a.T ? xs[lane * a.k_tiles + r.kb + i] : 0u;
          fence_async_shared();
          __syncwarp();
        }
        tc_fence_after();
        const uint64_t desc = sf_desc0 + (uint64_t)((stage * kFewSF) >> 4);
        const uint32_t tsf = tmem_base + 64 + 16 * stage;
        if (elect_one()) {
          tc_cp_32x128b_warpx4(tsf, desc);
          tc_cp_32x128b_warpx4(tsf + 4, desc + (uint64_t)(512 >> 4));
          tc_cp_32x128b_warpx4(tsf + 8, desc + (uint64_t)(1024 >> 4));
          tc_commit(smem_u32(full_bar + stage));
        }
        __syncwarp();
        ++nfill;
        if (++stage == a.stages) { stage = 0; phase ^= 1; }
      }
      s = r.next;
    }
    if (elect_one()) {
      tc_commit(smem_u32(drain_sf));   // every copy lands before TMEM is released
      mbar_wait_drain(smem_u32(drain_sf), 0);
      fills[2] = nfill;
    }
    __syncwarp();
  } else if (warp == 1 || warp == 12) {
    // ------------------------------------------------------------- MMA issuers, one per 128-row half
    const int h = warp == 12;
    const uint64_t desc0 = smem_desc(smem_u32(smem), 16, 1024, 2);
    int stage = 0, nfill = 0, nrun = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int s = s0; s < s1 && ok;) {
      const Run r = run_at(s);
      s = r.next;
      if (r.n == 0) continue;
      const int abuf = nrun & 1;
      const uint32_t acc_t = tmem_base + 32 * abuf + kFewRows * h;
      // the accumulator is free once the epilogue has drained the run before the last one
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(acc_empty + abuf), (uint32_t)(nrun >> 1 & 1) ^ 1u, a.status, abort_flag));
      if (!ok) break;
      auto run_steps = [&](auto shared) {   // compiled once for each kind
        for (int i = 0; i < r.n; ++i) {
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(full_bar + stage), phase, a.status, abort_flag));
          if (!ok) return;
          tc_fence_after();
          const uint64_t a_desc = desc0 + (uint64_t)((stage * kFewStage + h * 16384) >> 4);
          const uint64_t b_desc = desc0 + (uint64_t)((stage * kFewStage + kFewATile) >> 4);
          const uint32_t tsf = tmem_base + 64 + 16 * stage;
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t acc = i > 0 || j > 0;
              if constexpr (decltype(shared)::value)
                mma_bf16(acc_t, a_desc + (uint64_t)((32 * j) >> 4), b_desc + (uint64_t)((32 * j) >> 4), idesc_bf16(128, kFewRows), acc);
              else
                mma_mxf8f6f4(acc_t, a_desc + (uint64_t)((32 * j) >> 4), b_desc + (uint64_t)((32 * j) >> 4),
                             idesc_mx_e2m1_e4m3(128, kFewRows, j, j), (tsf + 4 * h) | ((uint32_t)j << 30),
                             (tsf + 8) | ((uint32_t)j << 30), acc);
            }
            tc_commit(smem_u32(empty_bar + stage));
          }
          __syncwarp();
          ++nfill;
          if (++stage == a.stages) { stage = 0; phase ^= 1; }
        }
      };
      if (MODE != FEW_LINEAR && r.shared) run_steps(std::true_type{});
      else run_steps(std::false_type{});
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
    const int et = tid - 64;   // 0 .. 255
    float* red = (float*)(smem + L.red);
    if constexpr (MODE == FEW_DOWN) {
      // the tokens' weights, while the first steps load; an expert that a token names twice counts
      // with the sum of both, in slot order
      for (int i = et; i < slots; i += 256) s_w[i] = __ldcg(a.w + i);
      few_bar();
      for (int i = et; i < used * a.T; i += 256) {
        const int e = elist[i / a.T], t = i % a.T;
        float w = 0.0f;
        for (int j = 0; j < a.k; ++j)
          if (s_idx[t * a.k + j] == e) w += s_w[t * a.k + j];
        hw[i] = w;
      }
      few_bar();
      griddep_wait();
    } else {
      uint32_t* xs = (uint32_t*)(smem + L.xs);
      for (int i = et; i < a.T * a.k_tiles; i += 256) xs[i] = ((const uint32_t*)a.xs)[i];
      asm volatile("bar.arrive 2, 288;" ::: "memory");
    }
    int nrun = 0;
    for (int s = s0; s < s1;) {
      // a segment: this CTA's runs of one tile
      float acc[kFewRows];
#pragma unroll
      for (int t = 0; t < kFewRows; ++t) acc[t] = 0.0f;
      const Run first = run_at(s);
      const int t0 = first.t0, t1 = min(t0 + first.len, s1);
      if (s > t0 + first.last) { s = t1; continue; }   // the tile's last step began in the CTA before
      const int from = s;
      const bool whole = from == t0 && t1 > t0 + first.last;
      while (s < t1) {
        const Run r = run_at(s);
        s = r.next;
        if (r.n == 0) continue;
        const int abuf = nrun & 1;
        int ok = 1;
        if (lane == 0) ok = mbar_wait(smem_u32(acc_full + abuf), (uint32_t)(nrun >> 1 & 1), a.status, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        tc_fence_after();
        uint32_t v[kFewRows];
        tmem_ld16(tmem_base + 32 * abuf + half * kFewRows + ((uint32_t)(q * 32) << 16), v);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(smem_u32(acc_empty + abuf));
        if (MODE == FEW_DOWN && !r.shared) {
          const int have = tokens[r.u];
#pragma unroll
          for (int t = 0; t < kFewRows; ++t)
            if (have >> t & 1) acc[t] = fmaf(hw[r.u * a.T + t], __uint_as_float(v[t]), acc[t]);
        } else {
#pragma unroll
          for (int t = 0; t < kFewRows; ++t) acc[t] += __uint_as_float(v[t]);
        }
        ++nrun;
      }
      bool finish = true;
      if (!whole) {
        // part of the tile's contraction: publish it; the last of the tile's CTAs adds them up
        float* mine = a.part + (size_t)(2 * c + (from == t0 ? 1 : 0)) * kFewPart + row;
#pragma unroll
        for (int t = 0; t < kFewRows; ++t)
          if (t < a.T) mine[t * 256] = acc[t];
        few_bar();
        // the CTAs with the tile's first and last step
        const int c_lo = cta_of(t0), c_hi = cta_of(t0 + first.last);
        if (et == 0) {
          // the CTA's partial ordered before the count, the others' partials after it
          const bool last = count_acq_rel(a.counters + c_lo) == (unsigned)(c_hi - c_lo);
          if (last) a.counters[c_lo] = 0;
          *s_last = last;
        }
        few_bar();
        finish = *s_last;
        if (finish) {
          // eight tokens and four CTAs at a time, so that the loads overlap (rows past T are loaded,
          // never used)
#pragma unroll
          for (int t8 = 0; t8 < kFewRows; t8 += 8) {
            if (t8 >= a.T) break;
            const float* p = a.part + (size_t)(2 * c_lo) * kFewPart + t8 * 256 + row;
            float v[8] = {};
            for (int i = c_lo; i <= c_hi; i += 4, p += 8 * kFewPart) {
              float n[4][8];
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int t = 0; t < 8; ++t)
                  n[j][t] = i + j <= c_hi ? __ldcg(p + (2 * j + (i + j == c_lo ? 1 : 0)) * kFewPart + t * 256) : 0.0f;
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int t = 0; t < 8; ++t) v[t] += n[j][t];
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) acc[t8 + t] = v[t];
          }
        }
      }
      if (finish) {
        if constexpr (MODE == FEW_GLU) {
          // the up half hands its values to the gate half, whose warps hold one 32-channel block each
          const int ch = row & 127;
          few_bar();
          if (half == 1) {
#pragma unroll
            for (int t = 0; t < kFewRows; ++t)
              if (t < a.T) red[t * 128 + ch] = acc[t];
          }
          few_bar();
          if (half == 0 && first.shared) {
            __nv_bfloat16* h = a.hsh + first.m * 128 + ch;
#pragma unroll
            for (int t = 0; t < kFewRows; ++t)
              if (t < a.T) h[(size_t)t * a.sh_tiles * 128] = __float2bfloat16_rn(glu_f<ACT>(acc[t], red[t * 128 + ch]));
          } else if (half == 0) {
            const int have = tokens[first.u];
            uint8_t* codes = a.hq + (size_t)first.u * a.T * a.m_tiles * 128 + first.m * 128 + ch;
            uint8_t* atom = a.hs + ((size_t)first.u * a.m_tiles + first.m) * 512 + q;
#pragma unroll
            for (int t = 0; t < kFewRows; ++t) {
              if (!(have >> t & 1)) continue;
              const float h = glu_f<ACT>(acc[t], red[t * 128 + ch]);
              const int e = mx_exp_e4m3(__reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7FFFFFFFu));
              const float v = h * __uint_as_float((uint32_t)(127 - e) << 23);
              codes[(size_t)t * a.m_tiles * 128] = (uint8_t)(f32x2_to_e4m3x2(v, 0.0f) & 0xFFu);
              if (lane == 0) atom[16 * t] = (uint8_t)(e + 127);
            }
          }
        } else {
          const int o_row = first.tile * 256 + row;
          if (o_row < a.rows) {
#pragma unroll
            for (int t = 0; t < kFewRows; ++t) {
              if (t >= a.T) break;
              const size_t o = (size_t)t * a.rows + o_row;
              if (MODE == FEW_LINEAR && a.y_f32) ((float*)a.y)[o] = acc[t];
              else ((__nv_bfloat16*)a.y)[o] = __float2bfloat16_rn(acc[t]);
            }
          }
        }
      }
    }
    if (MODE == FEW_DOWN && total == 0) {
      // every id was invalid, and no shared expert
      for (size_t i = (size_t)c * 256 + et; i < (size_t)a.T * a.rows; i += (size_t)gridDim.x * 256)
        ((__nv_bfloat16*)a.y)[i] = __float2bfloat16_rn(0.0f);
    }
  }
  __syncthreads();
  if (*abort_flag) {
    // a wait gave up: let the copies still in flight land before the CTA's shared memory is released
    if (tid == 0) {
      drain_ring(full_bar, a.stages, fills, 3, min(fills[3], fills[4]));
      drain_ring(sf_full, a.stages, fills, MODE == FEW_DOWN ? 2 : 1, fills[2]);
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kFewTmemCols);
  }
}

}  // namespace moe
