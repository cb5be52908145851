// The Muon step: momentum, orthogonalisation of the momentum by Newton-Schulz products, update.
//
//   M <- mu M + g, g = grad_scale R;  U0 = g + mu M (Nesterov) or M;  X = U0 / (||U0||_F + 1e-7);
//   steps times:  A = X X^T,  X <- a X + (b A + c A^2) X,  (a, b, c) = (3.4445, -4.7750, 2.0315);
//   W <- (1 - lr weight_decay) W - lr update_scale X.
// Every singular value of X goes through x <- a x + b x^3 + c x^5, which drives it towards 1; the
// singular vectors stay.  X is kept as [m, n] with m <= n (a tall matrix transposed), so that A is
// the smaller Gram matrix.
//
// The products run on the tensor cores in fp16 with fp32 accumulation: all values are at most
// about 1 here, so fp16's 11 bits serve where bf16 would keep 8.  Three choices keep five steps on a
// noisy gradient within 1e-3 of the exact iteration (3e-3 without them, 1.5e-2 with bf16 operands; a bf16
// result's own rounding is 1.7e-3):
//   - X is held as two fp16 planes, hi + lo 2^-11.  Products read hi; the term a X, by which small
//     singular values grow 3.4 times a step, uses both, so their rounding does not grow with them.
//   - b A and c A^2 use the same rounded A, so the polynomial is exact in the matrix that is stored.
//   - B = b A + c A^2 is stored less delta I, and a + delta multiplies X instead.  Near convergence
//     B is about -2.7 I; with delta the polynomial at the mean eigenvalue tr(A) / m, the large
//     diagonal stays in fp32 and only the small rest is rounded.
//
// The three products of a step are three launches of one engine (ns_kernel): the tcgen05 pipeline
// of umma_gemm_2sm.cuh with 256 x 256 tiles on SM pairs, or 128 x 128 tiles on single SMs where
// those would leave most SMs idle.  A and B are symmetric: only tiles on and above the diagonal
// are formed, and each is stored a second time transposed.
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

#include "embedding.cuh"
#include "ptx.cuh"
#include "simt.cuh"
#include "umma_gemm_2sm.cuh"

namespace dpclip {

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
constexpr double kNsEps = 1e-7;
constexpr float kLoScale = 2048.0f;  // the lo plane holds (x - hi) 2^11, a normal fp16 wherever hi is

enum NsKind : int { kNsGram = 0, kNsPoly = 1, kNsApply = 2 };
// Where kNsApply's result goes: the next step's planes; U in bf16, or W, as they lie or transposed.
enum NsOut : int { kNsPlanes = 0, kNsU = 1, kNsUT = 2, kNsW = 3, kNsWT = 4 };

struct alignas(64) NsParams {
  CUtensorMap tmA, tmB;
  int m, n;               // rows and columns of the result (kNsGram, kNsPoly: m x m)
  int tiles_m, tiles_n;   // tiles of the result; symmetric kinds: tiles_m on a side
  int num_units, k_blocks;
  const __half* A;        // kNsPoly: A
  const __half *hi, *lo;  // kNsApply: X
  __half *out, *out_lo;   // A or B; the next X's planes
  float* trace;           // one partial per 32 rows of A
  int order;              // rows of A (m of the iteration)
  int out_mode;           // NsOut
  __nv_bfloat16* U;
  float* W;
  float keep, rate;       // W <- keep W - rate X
  int early;              // at most half the SMs are used
  uint32_t* status;
};

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_nctaid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ uint4 pack_half8(const float* v) {
  uint4 q;
  __half2* h = reinterpret_cast<__half2*>(&q);
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
  return q;
}

__host__ __device__ constexpr uint32_t umma_idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4)                                 // D: f32; A and B format 0: f16
         | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// SPLIT: the CTAs of a cluster share one 128 x 128 tile of a symmetric product, each a run of its K
// blocks; each then adds up and stores the rows that it owns.  For products of few tiles and long K.
template <bool PAIR_, int KIND_, bool SPLIT_ = false>
struct NsConfig {
  static constexpr bool SPLIT = SPLIT_;
  static constexpr bool PAIR = PAIR_;
  static constexpr int KIND = KIND_;
  static constexpr int BM = 128;                       // rows a CTA
  static constexpr int TILE = PAIR ? 256 : 128;        // the tile is square
  static constexpr int BK = 64;
  static constexpr bool SYMMETRIC = KIND != kNsApply;
  static constexpr bool B_MN = KIND == kNsApply;       // X as [k, n]: its columns are contiguous
  static constexpr int OP_BYTES = BM * BK * 2;         // 16 KB of each operand a CTA and stage
  static constexpr int STAGE_BYTES = 2 * OP_BYTES;
  static constexpr int STAGES = SPLIT ? 4 : 6;
  static constexpr int NUM_BUFS = 2;
  static constexpr int THREADS = 320;                  // producer, MMA issuer, 8 epilogue warps
  // A block an epilogue warp; SPLIT: the parts of this CTA's rows, 128 x 128 fp32 in all.
  static constexpr int TURN_BYTES = SPLIT ? 128 * 128 * 4 : 8 * 32 * 33 * 4;
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + 256 + TURN_BYTES;
  static constexpr uint32_t IDESC = umma_idesc_f16(PAIR ? 256 : 128, TILE, false, B_MN);
  static_assert(SMEM_BYTES <= 232448, "dynamic shared memory per block");
  static_assert(!SPLIT || (SYMMETRIC && !PAIR), "split over K: symmetric products on single SMs");
};

struct NsUnit {
  int mb, nb;  // tile row and column
};

template <class Cfg>
__device__ __forceinline__ NsUnit ns_unit(const NsParams& p, int u) {
  NsUnit w;
  if constexpr (Cfg::SYMMETRIC) {  // pairs mb <= nb, row by row
    int row = 0;
    while (u >= p.tiles_m - row) {
      u -= p.tiles_m - row;
      ++row;
    }
    w.mb = row;
    w.nb = row + u;
  } else {  // groups of 8 row tiles, so that CTAs running together share operand tiles in L2
    constexpr int G = 8;
    const int per = G * p.tiles_n;
    const int first = (u / per) * G;
    const int rows = min(G, p.tiles_m - first);
    w.mb = first + (u % per) % rows;
    w.nb = (u % per) / rows;
  }
  return w;
}

// delta = b t + c t^2 at t = tr(A) / order, by every warp in the same order.
__device__ __forceinline__ float ns_delta(const float* __restrict__ trace, int order, uint32_t lane) {
  float t = 0.0f;
  for (int k = static_cast<int>(lane); k < (order + 31) / 32; k += 32) t += __ldcg(trace + k);
  t = warp_sum(t) / static_cast<float>(order);
  return t * fmaf(kNsC, t, kNsB);
}

// One epilogue warp's 32 x 32 block of kNsApply, turned through shared memory: X's planes and W are
// read, and everything is written, in runs of 64 to 128 bytes along the rows.  The planes' loads are a
// block ahead (the first before the accumulator is waited for), and no load stands behind a store (a row
// a lane, each load behind the store before it, the last product of a 4096 x 11008 update took 434 us).
// r0, col: the block's first row and column; cols: its columns in the matrix (0 .. 32, a multiple of 8).
struct NsPlanes {
  uint4 h[4], l[4];  // row 8 k + lane / 4, columns 8 (lane % 4) ..
};
__device__ __forceinline__ void ns_load_planes(const NsParams& p, int r0, int col, uint32_t lane, NsPlanes& x) {
  const int lr = static_cast<int>(lane) / 4, c = col + static_cast<int>(lane) % 4 * 8;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int row = r0 + 8 * k + lr;
    x.h[k] = x.l[k] = make_uint4(0u, 0u, 0u, 0u);
    if (row < p.m && c < p.n) {
      const long long at = static_cast<long long>(row) * p.n + c;
      x.h[k] = *reinterpret_cast<const uint4*>(p.hi + at);
      x.l[k] = *reinterpret_cast<const uint4*>(p.lo + at);
    }
  }
}
__device__ __forceinline__ void ns_apply_block(const NsParams& p, int r0, int col, int cols, uint32_t tacc,
                                               float (*turn)[33], uint32_t lane, float factor, const NsPlanes& old) {
  const int lr = static_cast<int>(lane) / 4, lc = static_cast<int>(lane) % 4 * 8;  // 8 rows of 4 x 8 columns
  {
    float v[32];
    __syncwarp();
    tmem_ld32(tacc, v);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) turn[lane][e] = v[e];
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // the new X, in place in the turned block
    const __half2* a = reinterpret_cast<const __half2*>(&old.h[k]);
    const __half2* b = reinterpret_cast<const __half2*>(&old.l[k]);
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(a[e]), g = __half22float2(b[e]);
      x[2 * e] = fmaf(factor, fmaf(g.x, 1.0f / kLoScale, f.x), turn[8 * k + lr][lc + 2 * e]);
      x[2 * e + 1] = fmaf(factor, fmaf(g.y, 1.0f / kLoScale, f.y), turn[8 * k + lr][lc + 2 * e + 1]);
    }
    const int row = r0 + 8 * k + lr;
    const bool in = row < p.m && lc < cols;
    const long long at = static_cast<long long>(row) * p.n + col + lc;
    if (p.out_mode == kNsPlanes) {
      uint4 h4, l4;
      __half2* nh = reinterpret_cast<__half2*>(&h4);
      __half2* nl = reinterpret_cast<__half2*>(&l4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        nh[e] = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
        const float2 f = __half22float2(nh[e]);
        nl[e] = __floats2half2_rn((x[2 * e] - f.x) * kLoScale, (x[2 * e + 1] - f.y) * kLoScale);
      }
      if (in && DP_DCHECK(at + 8 <= static_cast<long long>(p.m) * p.n, 60u, p.status)) {
        *reinterpret_cast<uint4*>(p.out + at) = h4;
        *reinterpret_cast<uint4*>(p.out_lo + at) = l4;
      }
    } else if (p.out_mode == kNsU) {
      uint4 pk;
      __nv_bfloat162* u = reinterpret_cast<__nv_bfloat162*>(&pk);
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      if (in) *reinterpret_cast<uint4*>(p.U + at) = pk;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) turn[8 * k + lr][lc + e] = x[e];
    }
  }
  if (p.out_mode == kNsPlanes || p.out_mode == kNsU) return;
  __syncwarp();
  if (p.out_mode == kNsW) {  // 4 rows of 8 float4 at a time
    float4 w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int row = r0 + 4 * k + static_cast<int>(lane) / 8, c = static_cast<int>(lane) % 8 * 4;
      w[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < p.m && c < cols) w[k] = *reinterpret_cast<const float4*>(p.W + static_cast<long long>(row) * p.n + col + c);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = 4 * k + static_cast<int>(lane) / 8, row = r0 + i, c = static_cast<int>(lane) % 8 * 4;
      if (row < p.m && c < cols)
        *reinterpret_cast<float4*>(p.W + static_cast<long long>(row) * p.n + col + c) =
            make_float4(fmaf(p.keep, w[k].x, -p.rate * turn[i][c]), fmaf(p.keep, w[k].y, -p.rate * turn[i][c + 1]),
                        fmaf(p.keep, w[k].z, -p.rate * turn[i][c + 2]), fmaf(p.keep, w[k].w, -p.rate * turn[i][c + 3]));
    }
    return;
  }
  // The caller's matrix is the transposed one: this block's columns are its rows, 32 of this block's
  // rows a run.
  const int row = r0 + static_cast<int>(lane);
  if (p.out_mode == kNsUT) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (row < p.m && e < cols) p.U[static_cast<long long>(col + e) * p.m + row] = __float2bfloat16_rn(turn[lane][e]);
    return;
  }
  float w[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) w[e] = row < p.m && e < cols ? p.W[static_cast<long long>(col + e) * p.m + row] : 0.0f;
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (row < p.m && e < cols)
      p.W[static_cast<long long>(col + e) * p.m + row] = fmaf(p.keep, w[e], -p.rate * turn[lane][e]);
}

// One epilogue warp's 32 x 32 block of A or B, turned through shared memory like X's: `product` gives
// this thread's 32 values of the product (row r0 + lane, columns col ..).  Rows and, off the diagonal,
// the same values as rows of the tile below it, are written in runs of 64 bytes.
template <class Cfg, typename Product>
__device__ __forceinline__ void ns_symmetric_block(const NsParams& p, const NsUnit& w, int r0, int col, int cols,
                                                   Product product, float (*turn)[33], uint32_t lane, float delta,
                                                   float& tr) {
  const int lr = static_cast<int>(lane) / 4, lc = static_cast<int>(lane) % 4 * 8;
  [[maybe_unused]] uint4 a4[4];
  if constexpr (Cfg::KIND == kNsPoly) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = r0 + 8 * k + lr;
      a4[k] = make_uint4(0u, 0u, 0u, 0u);
      if (row < p.m && lc < cols) a4[k] = *reinterpret_cast<const uint4*>(p.A + static_cast<long long>(row) * p.n + col + lc);
    }
  }
  {
    float v[32];
    product(v);
#pragma unroll
    for (int e = 0; e < 32; ++e) turn[lane][e] = v[e];
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = 8 * k + lr, row = r0 + i;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = turn[i][lc + e];
    if constexpr (Cfg::KIND == kNsPoly) {
      const __half2* h = reinterpret_cast<const __half2*>(&a4[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = __half22float2(h[e]);
        x[2 * e] = fmaf(kNsB, a.x, kNsC * x[2 * e]);
        x[2 * e + 1] = fmaf(kNsB, a.y, kNsC * x[2 * e + 1]);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (col + lc + e != row) continue;
      if constexpr (Cfg::KIND == kNsPoly)
        x[e] -= delta;
      else
        tr += x[e];
    }
    if constexpr (Cfg::KIND == kNsPoly) {
#pragma unroll
      for (int e = 0; e < 8; ++e) turn[i][lc + e] = x[e];
    }
    const long long at = static_cast<long long>(row) * p.n + col + lc;
    if (row < p.m && lc < cols && DP_DCHECK(at + 8 <= static_cast<long long>(p.m) * p.n, 62u, p.status))
      *reinterpret_cast<uint4*>(p.out + at) = pack_half8(x);
  }
  if (w.mb == w.nb) return;
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // column 8 k + lr of the block, its rows lc .. lc + 7
    const int i = 8 * k + lr;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = turn[lc + e][i];
    if (i < cols && r0 + lc < p.m)
      *reinterpret_cast<uint4*>(p.out + static_cast<long long>(col + i) * p.m + r0 + lc) = pack_half8(x);
  }
}

// This epilogue warp's share of a unit: 32 rows from r0, half the tile's columns.
template <class Cfg>
__device__ __forceinline__ void ns_epilogue(const NsParams& p, const NsUnit& w, int r0, uint32_t tacc, int half,
                                            float (*turn)[33], uint32_t lane, float delta, const NsPlanes& first) {
  float tr = 0.0f;
  [[maybe_unused]] NsPlanes ahead;
  if constexpr (Cfg::KIND == kNsApply) ahead = first;
#pragma unroll 1
  for (int c0 = half * (Cfg::TILE / 2); c0 < (half + 1) * (Cfg::TILE / 2); c0 += 32) {
    const int col = w.nb * Cfg::TILE + c0;
    const int cols = min(32, p.n - col);  // a multiple of 8
    if (cols <= 0) break;
    if constexpr (Cfg::KIND == kNsApply) {
      const NsPlanes old = ahead;
      if (c0 + 32 < (half + 1) * (Cfg::TILE / 2)) ns_load_planes(p, r0, col + 32, lane, ahead);
      ns_apply_block(p, r0, col, cols, tacc + c0, turn, lane, kNsA + delta, old);
    } else
      ns_symmetric_block<Cfg>(
          p, w, r0, col, cols,
          [&](float(&v)[32]) {
            __syncwarp();
            tmem_ld32(tacc + c0, v);
            tmem_ld_wait();
          },
          turn, lane, delta, tr);
    __syncwarp();
  }
  if constexpr (Cfg::KIND == kNsGram) {
    // The diagonal of these 32 rows lies in one half; rows past m were zero-filled and add nothing.
    if (w.mb == w.nb && (r0 - w.nb * Cfg::TILE) / (Cfg::TILE / 2) == half) {
      tr = warp_sum(tr);
      if (lane == 0 && r0 < p.m) p.trace[r0 / 32] = tr;
    }
  }
}

template <class Cfg>
__device__ __forceinline__ void ns_body(const NsParams& p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::STAGES * Cfg::STAGE_BYTES);
  uint64_t* full = bars;
  uint64_t* empty = bars + Cfg::STAGES;
  uint64_t* acc_full = bars + 2 * Cfg::STAGES;
  uint64_t* acc_empty = acc_full + Cfg::NUM_BUFS;
  uint64_t* drain = acc_empty + Cfg::NUM_BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  constexpr bool PAIR = Cfg::PAIR, SPLIT = Cfg::SPLIT;
  constexpr int kCtas = PAIR ? 2 : 1;
  const int warp = threadIdx.x / 32;
  const uint32_t lane = lane_id();
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  const bool leader = rank == 0;
  // SPLIT: one unit a cluster, whose CTA `share` of `shares` takes K blocks kb_begin .. kb_end.
  const int shares = SPLIT ? static_cast<int>(cluster_size()) : 1;
  const int share = SPLIT ? static_cast<int>(cluster_rank()) : 0;
  const int first = SPLIT ? blockIdx.x / shares : blockIdx.x / kCtas;
  const int step = SPLIT ? p.num_units : gridDim.x / kCtas;
  const int kb_share = (p.k_blocks + shares - 1) / shares;
  const int kb_begin = share * kb_share < p.k_blocks ? share * kb_share : p.k_blocks;
  const int kb_end = kb_begin + kb_share < p.k_blocks ? kb_begin + kb_share : p.k_blocks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(smem_addr(full + s), 1);
      mbar_init(smem_addr(empty + s), 1);
    }
    for (int b = 0; b < Cfg::NUM_BUFS; ++b) {
      mbar_init(smem_addr(acc_full + b), 1);
      mbar_init(smem_addr(acc_empty + b), 8 * kCtas);  // one arrival per epilogue warp of the tile
    }
    mbar_init(smem_addr(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_addr(tmem_slot), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_addr(tmem_slot), 512);
      tmem_relinquish();
    }
    tc_fence_before();
  }
  __syncthreads();
  if constexpr (PAIR || SPLIT) cluster_sync_all();  // every CTA runs, and its barriers exist, before remote accesses
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();  // barriers and TMEM are ready; global memory only from here
  // A launch that leaves SMs free lets the next one set up there meanwhile.
  if (p.early) griddep_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (every CTA)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      bool ok = true;
      for (int u = first; ok && u < p.num_units; u += step) {
        const NsUnit w = ns_unit<Cfg>(p, u);
        const int a0 = w.mb * Cfg::TILE + static_cast<int>(rank) * Cfg::BM;
        const int b0 = w.nb * Cfg::TILE + static_cast<int>(rank) * Cfg::BM;  // its half of B (PAIR), all of it else
        for (int kb = kb_begin; kb < kb_end; ++kb) {
          if (!mbar_wait_bounded(smem_addr(empty + stage), phase ^ 1u, abort_flag, p.status, 21u)) {
            ok = false;
            break;
          }
          const uint32_t sA = smem_addr(smem + stage * Cfg::STAGE_BYTES);
          const uint32_t sB = sA + Cfg::OP_BYTES;
          const int k0 = kb * Cfg::BK;
          if (leader) mbar_arrive_expect_tx(smem_addr(full + stage), kCtas * Cfg::STAGE_BYTES);
          if constexpr (PAIR) {
            const uint32_t bar = map_to_rank(smem_addr(full + stage), 0);
            tma_load_2d_pair(sA, &p.tmA, bar, k0, a0);
            if constexpr (Cfg::B_MN) {
              tma_load_2d_pair(sB, &p.tmB, bar, b0, k0);
              tma_load_2d_pair(sB + Cfg::BK * 128, &p.tmB, bar, b0 + 64, k0);
            } else {
              tma_load_2d_pair(sB, &p.tmB, bar, k0, b0);
            }
          } else {
            const uint32_t bar = smem_addr(full + stage);
            tma_load_2d(sA, &p.tmA, bar, k0, a0);
            if constexpr (Cfg::B_MN) {
              tma_load_2d(sB, &p.tmB, bar, b0, k0);
              tma_load_2d(sB + Cfg::BK * 128, &p.tmB, bar, b0 + 64, k0);
            } else {
              tma_load_2d(sB, &p.tmB, bar, k0, b0);
            }
          }
          if (++stage == Cfg::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          ++issued;
        }
      }
      // No copy may still write shared memory when the CTA leaves (or SPLIT uses it again), not even after
      // a wait elsewhere ran out.  The pair's copies arrive at the leader, and its peer leaves after it.
      const unsigned long long t0 = global_timer_ns();
      for (int k = 0; leader && k < Cfg::STAGES && k < issued; ++k) {
        stage = stage > 0 ? stage - 1 : Cfg::STAGES - 1;
        if (stage == Cfg::STAGES - 1) phase ^= 1u;
        while (!mbar_try_wait(smem_addr(full + stage), phase) && global_timer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    if (leader && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int buf = 0;
      uint32_t buf_phase = 0;
      bool ok = true;
      for (int u = first; ok && u < p.num_units; u += step) {
        if (!mbar_wait_bounded(smem_addr(acc_empty + buf), buf_phase ^ 1u, abort_flag, p.status, 22u)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + buf * 256;
        for (int kb = kb_begin; kb < kb_end; ++kb) {
          if (!mbar_wait_bounded(smem_addr(full + stage), phase, abort_flag, p.status, 23u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sA = smem_addr(smem + stage * Cfg::STAGE_BYTES);
          const uint32_t sB = sA + Cfg::OP_BYTES;
#pragma unroll
          for (int ks = 0; ks < Cfg::BK / 16; ++ks) {
            const uint64_t da = umma_desc_sw128(sA + ks * 32, 16, 1024);
            const uint64_t db = Cfg::B_MN ? umma_desc_sw128(sB + ks * 2048, Cfg::BK * 128, 1024)
                                          : umma_desc_sw128(sB + ks * 32, 16, 1024);
            // (These issue tcgen05.mma kind::f16; the instruction descriptor says fp16 operands.)
            if constexpr (PAIR)
              umma_bf16_pair(d_tmem, da, db, Cfg::IDESC, (kb > kb_begin || ks > 0) ? 1u : 0u);
            else
              umma_bf16(d_tmem, da, db, Cfg::IDESC, (kb > kb_begin || ks > 0) ? 1u : 0u);
          }
          if constexpr (PAIR)
            umma_commit_pair(smem_addr(empty + stage), 0x3);
          else
            umma_commit(smem_addr(empty + stage));
          if (++stage == Cfg::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if constexpr (PAIR)
          umma_commit_pair(smem_addr(acc_full + buf), 0x3);
        else
          umma_commit(smem_addr(acc_full + buf));
        if (++buf == Cfg::NUM_BUFS) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
      // No MMA may still write TMEM when it is released.
      if constexpr (PAIR)
        umma_commit_pair_local(smem_addr(drain));
      else
        umma_commit(smem_addr(drain));
      const unsigned long long t0 = global_timer_ns();
      while (!mbar_try_wait(smem_addr(drain), 0u)) {
        if (global_timer_ns() - t0 > kWaitLimitNs) {
          if (p.status) atomicCAS(p.status, 0u, 25u);
          break;
        }
      }
    }
  } else if constexpr (SPLIT) {
    // ------------------------------------------------------------ this CTA's part of the tile to the owners
    const int wq = warp & 3, half = (warp - 2) >> 2;
    const bool ok = mbar_wait_warp(smem_addr(acc_full), 0u, abort_flag, p.status, 24u);
    tc_fence_after();
    const int rows = 128 / shares, owner = 32 * wq / rows, row = 32 * wq % rows + static_cast<int>(lane);
    // parts[share][column][row]: a column of the warp's 32 rows is 128 contiguous bytes.
    const uint32_t to = map_to_rank(smem_addr(smem + Cfg::STAGES * Cfg::STAGE_BYTES + 256), owner) +
                        static_cast<uint32_t>((share * 128 + 64 * half) * rows + row) * 4u;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      float v[32];
      __syncwarp();
      tmem_ld32(tmem_base + (static_cast<uint32_t>(wq * 32) << 16) + 64 * half + 32 * part, v);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 32; ++e)
        st_cluster_f32(to + static_cast<uint32_t>((32 * part + e) * rows) * 4u, ok && kb_end > kb_begin ? v[e] : 0.0f);
    }
    tc_fence_before();
  } else {
    // ------------------------------------------------------------ epilogue warps 2..9 (every CTA)
    const int wq = warp & 3;           // TMEM lane quarter this warp may access
    const int half = (warp - 2) >> 2;  // and its half of the columns
    float(*const turn)[33] = reinterpret_cast<float(*)[33]>(smem + Cfg::STAGES * Cfg::STAGE_BYTES + 256) + 32 * (warp - 2);
    const float delta = Cfg::KIND == kNsGram ? 0.0f : ns_delta(p.trace, p.order, lane);
    int buf = 0;
    uint32_t buf_phase = 0;
    for (int u = first; u < p.num_units; u += step) {
      const NsUnit w = ns_unit<Cfg>(p, u);
      const int r0 = w.mb * Cfg::TILE + static_cast<int>(rank) * Cfg::BM + wq * 32;
      NsPlanes planes;
      if constexpr (Cfg::KIND == kNsApply) ns_load_planes(p, r0, w.nb * Cfg::TILE + half * (Cfg::TILE / 2), lane, planes);
      if (!mbar_wait_warp(smem_addr(acc_full + buf), buf_phase, abort_flag, p.status, 24u)) break;
      tc_fence_after();
      const uint32_t tacc = tmem_base + buf * 256 + (static_cast<uint32_t>(wq * 32) << 16);
      ns_epilogue<Cfg>(p, w, r0, tacc, half, turn, lane, delta, planes);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          mbar_arrive_remote(map_to_rank(smem_addr(acc_empty + buf), 0));
        else
          mbar_arrive(smem_addr(acc_empty + buf));
      }
      if (++buf == Cfg::NUM_BUFS) {
        buf = 0;
        buf_phase ^= 1u;
      }
    }
  }
  if constexpr (SPLIT) {
    __syncthreads();
    cluster_sync_all();  // every part of this CTA's rows has arrived, and nothing is sent after it
    const int rows = 128 / shares, ew = warp - 2;
    // 32 x 32 blocks of the owned rows, one a warp: rows / 32 x 4 of them, at most 8.
    if (ew >= 0 && ew < rows / 32 * 4) {
      const NsUnit w = ns_unit<Cfg>(p, first);
      const int rb = ew / 4 * 32, c0 = ew % 4 * 32;
      const int r0 = w.mb * 128 + share * rows + rb, col = w.nb * 128 + c0, cols = min(32, p.n - col);
      const float* parts = reinterpret_cast<const float*>(smem + Cfg::STAGES * Cfg::STAGE_BYTES + 256);
      const float delta = Cfg::KIND == kNsGram ? 0.0f : ns_delta(p.trace, p.order, lane);
      float tr = 0.0f;
      if (cols > 0)
        ns_symmetric_block<Cfg>(
            p, w, r0, col, cols,
            [&](float(&v)[32]) {
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = 0.0f;
              for (int s = 0; s < shares; ++s)
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] += parts[(s * 128 + c0 + e) * rows + rb + static_cast<int>(lane)];
            },
            reinterpret_cast<float(*)[33]>(smem) + 32 * ew, lane, delta, tr);  // the ring's stages are free
      __syncwarp();
      if (Cfg::KIND == kNsGram && r0 == col) {  // the block on the diagonal
        tr = warp_sum(tr);
        if (lane == 0 && r0 < p.m) p.trace[r0 / 32] = tr;
      }
    }
  }
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // no CTA leaves while its peer may still signal it
  griddep_launch_dependents();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem_base, 512);
    else
      tmem_dealloc(tmem_base, 512);
  }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1) ns_kernel(const __grid_constant__ NsParams p) {
  ns_body<Cfg>(p);
}
template <class Cfg>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg::THREADS, 1)
    ns_pair_kernel(const __grid_constant__ NsParams p) {
  ns_body<Cfg>(p);
}

// ------------------------------------------------------------------------ one launch, m <= 128
// The whole iteration of a matrix with at most 128 rows (as m x n), such as a projected gradient of
// r = 128, in one cluster.  Every CTA keeps up to 256 columns of X: in fp32 in TMEM, and their fp16
// part as a shared-memory tile that serves both products (K-major for X X^T, MN-major for B X).  A step:
//   each CTA forms X X^T of its columns; the CTAs add their parts (each the rows it owns, sent as
//   columns: the matrix is symmetric, and so a warp's 32 lanes write 128 contiguous bytes; read by the
//   owner instead, a step took 12 us) and send the rounded rows of A to all; each forms B, and then its
//   columns of the next X.
// A step is then about 8 us of latency with several CTAs (half of it the exchange) and 4 us with one,
// against 18 us as three launches: 1024 x 128, five steps, 52 us against 105.
// Exact in the same places as the products above (X in fp32 where those keep two fp16 planes).

// Registers to 32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_16(uint32_t addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

struct NsSmall {
  const void* R;
  const float* M;
  int rows, cols;  // as the caller has them; m, n: the smaller and the larger
  int m, n;
  float mu, gs;
  int nesterov;
  const double* partials;  // of the momentum's squared norm
  int count;
  int steps;
  int chunks;              // 64-column chunks of X a CTA keeps, at most 4
  __nv_bfloat16* U;        // or
  float* W;                // W <- keep W - rate X
  float keep, rate;
  uint32_t* status;
};

constexpr int kNsSmallThreads = 256;
constexpr int kNsSmallRows = 128;
constexpr int kNsSmallMaxChunks = 4;
constexpr int kNsSmallCtas = 16;      // at most (more than 8 where the device takes such clusters)
constexpr int kNsTile = kNsSmallRows * 128;  // bytes of a 128 x 64 fp16 tile
constexpr int kNsSmallSmem = 1024 + (kNsSmallMaxChunks + 4) * kNsTile + kNsSmallRows * kNsSmallRows * 4;

// 16-byte unit `unit` (of 8) of row r in a 128-byte-swizzled tile.
__device__ __forceinline__ uint32_t ns_unit_offset(int r, int unit) {
  return static_cast<uint32_t>(r * 128 + ((unit ^ (r & 7)) << 4));
}

template <typename T, bool MUON>
__global__ void __launch_bounds__(kNsSmallThreads, 1) ns_small_kernel(const __grid_constant__ NsSmall p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ float diag[kNsSmallRows];
  __shared__ double norm_part[kNsSmallThreads / 32];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const hi = smem;                                   // X: [chunk][128][64]
  uint8_t* const sA = hi + kNsSmallMaxChunks * kNsTile;       // A, and B below: [2][128][64]
  uint8_t* const sB = sA + 2 * kNsTile;
  float* const recv = reinterpret_cast<float*>(sB + 2 * kNsTile);  // [CTA][owned row][128] parts of A

  const int tid = threadIdx.x, warp = tid / 32, half = warp / 4;
  const uint32_t lane = lane_id();
  const int r = 32 * (warp % 4) + static_cast<int>(lane);  // this thread's row (TMEM lane)
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const int owned = kNsSmallRows / static_cast<int>(ctas);  // rows of A a CTA adds up, a power of two
  const int owned_bits = 31 - __clz(owned);
  const int chunk0 = static_cast<int>(rank) * p.chunks;
  const int chunks = max(0, min(p.chunks, (p.n + 63) / 64 - chunk0));

  if (tid == 0) {
    mbar_init(smem_addr(&done), 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    __syncwarp();
    tmem_alloc(smem_addr(&tmem_slot), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  if (ctas > 1) cluster_sync_all();  // every CTA runs before its shared memory is written from others
  tc_fence_after();
  const uint32_t tm_x = tmem_slot + (static_cast<uint32_t>(32 * (warp % 4)) << 16);  // X, 256 columns
  const uint32_t tm_acc = tm_x + 256;                                                // the product at hand
  const uint32_t acc0 = tmem_slot + 256;
  griddep_wait();

  // 1 / (||u|| + eps), in the same order in every CTA.
  double s = 0.0;
  for (int k = tid; k < p.count; k += kNsSmallThreads) s += p.partials[k];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (lane == 0) norm_part[warp] = s;
  __syncthreads();
  s = 0.0;
  for (int w = 0; w < kNsSmallThreads / 32; ++w) s += norm_part[w];
  const double inv = 1.0 / (sqrt(s) + kNsEps);

  const bool tall = p.rows > p.cols;
  // X at 32 places: all loads first (a place outside the matrix reads element 0), then the arithmetic.
  auto values = [&](auto place, float (&v)[32]) {
    float x[32];
    [[maybe_unused]] float mo[MUON ? 32 : 1];
    bool in[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const long long at = place(j);
      in[j] = at >= 0;
      x[j] = static_cast<float>(static_cast<const T*>(p.R)[in[j] ? at : 0]);
      if constexpr (MUON) mo[j] = p.M[in[j] ? at : 0];
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      float u = x[j];
      if constexpr (MUON) u = p.nesterov ? fmaf(p.mu, mo[j], p.gs * x[j]) : mo[j];
      v[j] = in[j] ? static_cast<float>(static_cast<double>(u) * inv) : 0.0f;
    }
  };
  // Element (row, c) of the m x n matrix in the caller's, -1 outside.
  auto place_of = [&](int row, int c) -> long long {
    if (row >= p.m || c >= p.n) return -1;
    return tall ? static_cast<long long>(c) * p.cols + row : static_cast<long long>(row) * p.cols + c;
  };
  auto put_hi = [&](int cc, const float (&v)[32]) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<uint4*>(hi + cc * kNsTile + ns_unit_offset(r, 4 * half + q)) = pack_half8(v + 8 * q);
  };
  // A wide matrix is read and written by rows: a warp's 32 x 32 block is turned in shared memory (the
  // tiles of A and B, which hold nothing then).  A tall one already lies as the lanes hold it.
  float(*const turn)[33] = reinterpret_cast<float(*)[33]>(sA) + 32 * warp;
  for (int cc = 0; cc < chunks; ++cc) {
    float v[32];
    const int col = (chunk0 + cc) * 64 + 32 * half;
    if (tall) {
      values([&](int j) { return place_of(r, col + j); }, v);
    } else {
      values([&](int j) { return place_of(32 * (warp % 4) + j, col + static_cast<int>(lane)); }, v);
#pragma unroll
      for (int j = 0; j < 32; ++j) turn[j][lane] = v[j];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = turn[lane][j];
      __syncwarp();
    }
    __syncwarp();
    tmem_st32(tm_x + 64 * cc + 32 * half, v);
    put_hi(cc, v);
  }
  __syncwarp();
  tmem_st_wait();

  uint32_t parity = 0;
  // Ends a phase of shared-memory writes and TMEM accesses, lets thread 0 issue MMAs, waits for them.
  // A wait that runs out is recorded and the steps go on: every barrier is still met by every thread.
  auto multiply = [&](auto issue) {
    fence_async_proxy();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      fence_async_proxy();
      issue();
      umma_commit(smem_addr(&done));
    }
    __syncwarp();
    mbar_wait_warp(smem_addr(&done), parity, &abort_word, p.status, 41u);
    parity ^= 1u;
    tc_fence_after();
  };
  constexpr uint32_t kSquare = umma_idesc_f16(128, 128, false, false);

  for (int step = 0; step < p.steps; ++step) {
    // A = X X^T over this CTA's columns.
    multiply([&] {
      for (int cc = 0; cc < chunks; ++cc)
        for (int ks = 0; ks < 4; ++ks) {
          const uint64_t x = umma_desc_sw128(smem_addr(hi) + cc * kNsTile + ks * 32, 16, 1024);
          umma_bf16(acc0, x, x, kSquare, (cc > 0 || ks > 0) ? 1u : 0u);
        }
    });
    if (ctas == 1) {
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        float v[32];
        __syncwarp();
        tmem_ld32(tm_acc + 64 * half + 32 * part, v);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(sA + half * kNsTile + ns_unit_offset(r, 4 * part + q)) = pack_half8(v + 8 * q);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (64 * half + 32 * part + e == r) diag[r] = v[e];
      }
    } else {
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        float v[32];
        __syncwarp();
        tmem_ld32(tm_acc + 64 * half + 32 * part, v);
        tmem_ld_wait();
        const int c0 = 64 * half + 32 * part;
#pragma unroll
        for (int e = 0; e < 32; ++e) {  // row c0 + e of A, column r
          const int owner = (c0 + e) >> owned_bits, row = (c0 + e) & (owned - 1);
          st_cluster_f32(map_to_rank(smem_addr(recv + (static_cast<int>(rank) * owned + row) * kNsSmallRows + r), owner),
                         chunks > 0 ? v[e] : 0.0f);
        }
      }
      __syncwarp();
      cluster_sync_all();
      for (int unit = tid; unit < owned * (kNsSmallRows / 8); unit += kNsSmallThreads) {
        const int row = unit / (kNsSmallRows / 8), col = unit % (kNsSmallRows / 8) * 8;
        float v[8] = {};
        for (uint32_t c = 0; c < ctas; ++c) {
          const float4* in = reinterpret_cast<const float4*>(recv + (static_cast<int>(c) * owned + row) * kNsSmallRows + col);
          const float4 a = in[0], b = in[1];
          v[0] += a.x;
          v[1] += a.y;
          v[2] += a.z;
          v[3] += a.w;
          v[4] += b.x;
          v[5] += b.y;
          v[6] += b.z;
          v[7] += b.w;
        }
        const int R = static_cast<int>(rank) * owned + row;
        const uint32_t at = smem_addr(sA) + (col / 64) * kNsTile + ns_unit_offset(R, (col % 64) / 8);
        const uint4 q = pack_half8(v);
        for (uint32_t c = 0; c < ctas; ++c) st_cluster_16(map_to_rank(at, c), q);
        if (R >= col && R < col + 8) {
          float d = v[0];
#pragma unroll
          for (int e = 1; e < 8; ++e) d = R == col + e ? v[e] : d;
          for (uint32_t c = 0; c < ctas; ++c) st_cluster_f32(map_to_rank(smem_addr(diag + R), c), d);
        }
      }
      fence_async_proxy();
      __syncwarp();
      cluster_sync_all();
    }
    // A^2, then B = b A + c A^2 - delta I.
    multiply([&] {
      for (int ks = 0; ks < 8; ++ks) {
        const uint64_t a = umma_desc_sw128(smem_addr(sA) + (ks / 4) * kNsTile + (ks % 4) * 32, 16, 1024);
        umma_bf16(acc0, a, a, kSquare, ks > 0 ? 1u : 0u);
      }
    });
    float tr = 0.0f;
#pragma unroll
    for (int k = 0; k < kNsSmallRows / 32; ++k) tr += diag[32 * k + lane];  // rows past m are zero
    tr = warp_sum(tr) / static_cast<float>(p.m);
    const float delta = tr * fmaf(kNsC, tr, kNsB);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      float v[32];
      __syncwarp();
      tmem_ld32(tm_acc + 64 * half + 32 * part, v);
      tmem_ld_wait();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t at = half * kNsTile + ns_unit_offset(r, 4 * part + q);
        const uint4 a4 = *reinterpret_cast<const uint4*>(sA + at);
        const __half2* h = reinterpret_cast<const __half2*>(&a4);
        float b[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = __half22float2(h[e]);
          b[2 * e] = fmaf(kNsB, a.x, kNsC * v[8 * q + 2 * e]);
          b[2 * e + 1] = fmaf(kNsB, a.y, kNsC * v[8 * q + 2 * e + 1]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (64 * half + 32 * part + 8 * q + e == r) b[e] -= delta;
        *reinterpret_cast<uint4*>(sB + at) = pack_half8(b);
      }
    }
    // X = (a + delta) X + B X.
    const uint32_t wide = umma_idesc_f16(128, 64 * max(chunks, 1), false, true);
    multiply([&] {
      if (chunks > 0)
        for (int ks = 0; ks < 8; ++ks)
          umma_bf16(acc0, umma_desc_sw128(smem_addr(sB) + (ks / 4) * kNsTile + (ks % 4) * 32, 16, 1024),
                    umma_desc_sw128(smem_addr(hi) + ks * 2048, kNsTile, 1024), wide, ks > 0 ? 1u : 0u);
    });
    const bool last = step + 1 == p.steps;
    for (int cc = 0; cc < chunks; ++cc) {
      float v[32], x[32];
      __syncwarp();
      tmem_ld32(tm_acc + 64 * cc + 32 * half, v);
      tmem_ld32(tm_x + 64 * cc + 32 * half, x);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = fmaf(kNsA + delta, x[j], v[j]);
      if (!last) {
        __syncwarp();
        tmem_st32(tm_x + 64 * cc + 32 * half, v);
        put_hi(cc, v);
        continue;
      }
      const int col = (chunk0 + cc) * 64 + 32 * half;
      auto write = [&](auto place) {
        float w[32];
        if (!p.U) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const long long at = place(j);
            w[j] = p.W[at >= 0 ? at : 0];
          }
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const long long at = place(j);
          if (at < 0 || !DP_DCHECK(in_buffer(at, 1, static_cast<long long>(p.rows) * p.cols), 61u, p.status)) continue;
          if (p.U)
            p.U[at] = __float2bfloat16_rn(v[j]);
          else
            p.W[at] = fmaf(p.keep, w[j], -p.rate * v[j]);
        }
      };
      if (tall) {
        write([&](int j) { return place_of(r, col + j); });
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) turn[lane][j] = v[j];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = turn[j][lane];
        __syncwarp();
        write([&](int j) { return place_of(32 * (warp % 4) + j, col + static_cast<int>(lane)); });
      }
    }
    __syncwarp();
    tmem_st_wait();
  }
  // Every MMA was waited for; after a wait that ran out one may still be at work.
  __syncthreads();
  griddep_launch_dependents();
  if (tid == 0 && abort_word) {
    umma_commit(smem_addr(&done));
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait(smem_addr(&done), parity) && global_timer_ns() - t0 < kWaitLimitNs) {
    }
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_slot, 512);
  }
}

// ------------------------------------------------------------------------------ around them
constexpr int kMuonThreads = 256;

// MUON: M <- mu M + gs R, and u = gs R + mu M (nesterov) or M; else u = R.  Block partials of
// sum u^2, in fp64 (the squares of large or tiny gradients leave fp32's range).
template <typename T, bool MUON>
__global__ void __launch_bounds__(kMuonThreads)
    muon_momentum_kernel(const T* __restrict__ R, float* __restrict__ M, long long vecs, float mu, float gs,
                         int nesterov, double* __restrict__ partials, uint32_t* __restrict__ status) {
  griddep_enter();
  constexpr int V = EmbVec<T>::N;
  __shared__ double part[kMuonThreads / 32];
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0u;
  const long long stride = static_cast<long long>(gridDim.x) * kMuonThreads;
  double ss = 0.0;
  constexpr int kU = 4;
  for (long long v0 = static_cast<long long>(blockIdx.x) * kMuonThreads + threadIdx.x; v0 < vecs; v0 += kU * stride) {
    uint4 q[kU], qm[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      if (v0 + k * stride >= vecs) continue;
      q[k] = __ldg(reinterpret_cast<const uint4*>(R) + v0 + k * stride);
      if constexpr (MUON) qm[k] = reinterpret_cast<const uint4*>(M)[v0 + k * stride];
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      if (v0 + k * stride >= vecs) continue;
      float u[V];
      unpack16(q[k], u, R);
      if constexpr (MUON) {
        float m[4];
        unpack16(qm[k], m, M);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float g = gs * u[e];
          m[e] = fmaf(mu, m[e], g);
          u[e] = nesterov ? fmaf(mu, m[e], g) : m[e];
        }
        reinterpret_cast<uint4*>(M)[v0 + k * stride] =
            make_uint4(__float_as_uint(m[0]), __float_as_uint(m[1]), __float_as_uint(m[2]), __float_as_uint(m[3]));
      }
#pragma unroll
      for (int e = 0; e < V; ++e) ss = fma(static_cast<double>(u[e]), static_cast<double>(u[e]), ss);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = ss;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kMuonThreads / 32; ++w) s += part[w];
    partials[blockIdx.x] = s;
  }
}

// 1 / (sqrt(sum of the partials) + eps), by every block in the same order.
__device__ __forceinline__ double muon_inverse_norm(const double* __restrict__ partials, int count) {
  __shared__ double part[kMuonThreads / 32];
  double s = 0.0;
  for (int k = threadIdx.x; k < count; k += kMuonThreads) s += partials[k];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = s;
  __syncthreads();
  s = 0.0;
  for (int w = 0; w < kMuonThreads / 32; ++w) s += part[w];
  return 1.0 / (sqrt(s) + kNsEps);
}

// The planes of X = u / (||u|| + eps): 64 x 64 tiles through shared memory when the matrix is tall
// (TRANSPOSE: X[c, r] = u[r, c]), straight through registers otherwise.
template <typename T, bool MUON, bool TRANSPOSE>
__global__ void __launch_bounds__(kMuonThreads)
    muon_prepare_kernel(const T* __restrict__ R, const float* __restrict__ M, int rows, int cols, float mu, float gs,
                        int nesterov, const double* __restrict__ partials, int count, __half* __restrict__ hi,
                        __half* __restrict__ lo) {
  griddep_enter();
  const double inv = muon_inverse_norm(partials, count);
  auto value = [&](long long at) {
    float u;
    if constexpr (MUON) {
      const float m = M[at];
      u = nesterov ? fmaf(mu, m, gs * static_cast<float>(R[at])) : m;
    } else {
      u = static_cast<float>(R[at]);
    }
    return static_cast<float>(static_cast<double>(u) * inv);
  };
  auto put = [&](long long at, float a, float b) {  // two neighbours
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    *reinterpret_cast<__half2*>(hi + at) = h;
    *reinterpret_cast<__half2*>(lo + at) = __floats2half2_rn((a - f.x) * kLoScale, (b - f.y) * kLoScale);
  };
  if constexpr (TRANSPOSE) {
    __shared__ float tile[64][65];
    const int tc = (cols + 63) / 64;
    const long long tiles = static_cast<long long>((rows + 63) / 64) * tc;
    for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
      const int r0 = static_cast<int>(t / tc) * 64, c0 = static_cast<int>(t % tc) * 64;
      for (int k = threadIdx.x; k < 64 * 64; k += kMuonThreads) {
        const int r = r0 + k / 64, c = c0 + k % 64;
        tile[k / 64][k % 64] = r < rows && c < cols ? value(static_cast<long long>(r) * cols + c) : 0.0f;
      }
      __syncthreads();
      for (int k = threadIdx.x; k < 64 * 32; k += kMuonThreads) {
        const int c = c0 + k / 32, r = r0 + 2 * (k % 32);  // rows come in multiples of 8
        if (c < cols && r < rows)
          put(static_cast<long long>(c) * rows + r, tile[2 * (k % 32)][k / 32], tile[2 * (k % 32) + 1][k / 32]);
      }
      __syncthreads();
    }
  } else {
    const long long pairs = static_cast<long long>(rows) * cols / 2;
    const long long stride = static_cast<long long>(gridDim.x) * kMuonThreads;
#pragma unroll 4
    for (long long k = static_cast<long long>(blockIdx.x) * kMuonThreads + threadIdx.x; k < pairs; k += stride)
      put(2 * k, value(2 * k), value(2 * k + 1));
  }
}

}  // namespace dpclip
