// RMS norm with the residual's addition, its backward, and the privatised gradient of its gain.
//
//   h = round(x + res),  r = 1 / sqrt(mean_j h_j^2 + eps),  y_j = h_j r g_j;
//   backward, u_j = g_j dy_j:  dh_j = r (u_j - h_j r mean_k(u_k h_k r))  (+ the gradient that
//   reaches h past the norm);
//   sample i's gain gradient  g_i[j] = sum_t dy_tj h_tj r_t,  n_i = ||g_i||,
//   S[j] = sum_i c_i g_i[j] + sigma C z_j.
// r is formed again in the backward from the row it reads anyway, so nothing but h is kept.
// Every sum of a row or a column is in fp32, the sums over samples and norms in fp64, all in a
// fixed order: the bits repeat.
//
// A row is held in registers, so it is read once, and its two sums (h^2 and u h) are one reduction.
// Columns stay with their thread, so the gain's values and the gain gradient's sums live in registers
// across the rows of a block.  Both kernels are bound by HBM.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "embedding.cuh"
#include "ptx.cuh"
#include "rng.cuh"
#include "simt.cuh"

namespace dpclip {

template <typename T, int V>
__device__ __forceinline__ uint4 pack16(const float (&f)[V], const T*) {
  uint4 q;
  if constexpr (sizeof(T) == 2) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
  } else {
    q = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  return q;
}

// Sums a and b over the kTpr threads of a row.  More than a warp: through shared memory, two
// slots in turn so that one barrier a row is enough (a slot is written again only after every
// thread has passed the barrier of the row between).
template <int kTpr>
__device__ __forceinline__ void row_sums(float& a, float& b, float (*red)[2][kTpr / 32 > 0 ? kTpr / 32 : 1], int turn) {
  a = warp_sum(a);
  b = warp_sum(b);
  if constexpr (kTpr > 32) {
    const int warp = threadIdx.x / 32;
    if (threadIdx.x % 32 == 0) {
      red[turn][0][warp] = a;
      red[turn][1][warp] = b;
    }
    __syncthreads();
    a = 0.0f;
    b = 0.0f;
#pragma unroll
    for (int w = 0; w < kTpr / 32; ++w) {
      a += red[turn][0][w];
      b += red[turn][1][w];
    }
  }
}

// One row per kTpr threads, kNv vectors of 16 bytes each; a block of kThreads threads takes kThreads / kTpr rows at a time.
template <typename T, int kTpr, int kNv, bool RES>
__global__ void __launch_bounds__(kTpr < 128 ? 128 : kTpr)
    rmsnorm_kernel(const T* __restrict__ X, const T* __restrict__ res, const float* __restrict__ gain, long long rows,
                   int d, float eps, T* __restrict__ H, T* __restrict__ Y) {
  griddep_enter();
  constexpr int V = EmbVec<T>::N;
  constexpr int kThreads = kTpr < 128 ? 128 : kTpr;
  constexpr int kRows = kThreads / kTpr;
  __shared__ float red[2][2][kTpr / 32 > 0 ? kTpr / 32 : 1];
  const int t = threadIdx.x % kTpr;
  const int vecs = d / V;
  const float inv_d = 1.0f / static_cast<float>(d);
  int turn = 0;
  // kRows > 1 only with a warp per row: no barrier then, so warps may run out of rows alone.
  for (long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / kTpr; row < rows;
       row += static_cast<long long>(gridDim.x) * kRows, turn ^= 1) {
    const uint4* x = reinterpret_cast<const uint4*>(X + row * d);
    const uint4* r = RES ? reinterpret_cast<const uint4*>(res + row * d) : nullptr;
    uint4 q[kNv], qr[kNv];
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      q[k] = qr[k] = make_uint4(0u, 0u, 0u, 0u);
      if (t + k * kTpr < vecs) {
        q[k] = __ldg(x + t + k * kTpr);
        if constexpr (RES) qr[k] = __ldg(r + t + k * kTpr);
      }
    }
    float ss = 0.0f, none = 0.0f;
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      float f[V];
      unpack16(q[k], f, X);
      if constexpr (RES) {
        float e[V];
        unpack16(qr[k], e, X);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] += e[j];
        q[k] = pack16<T, V>(f, X);  // h as its backward will read it; the norm is of that
        unpack16(q[k], f, X);
        if (t + k * kTpr < vecs) reinterpret_cast<uint4*>(H + row * d)[t + k * kTpr] = q[k];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(f[j], f[j], ss);
    }
    row_sums<kTpr>(ss, none, red, turn);
    const float inv = 1.0f / sqrtf(fmaf(ss, inv_d, eps));
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      if (t + k * kTpr >= vecs) continue;
      float f[V];
      unpack16(q[k], f, X);
      const float4* g = reinterpret_cast<const float4*>(gain + static_cast<long long>(t + k * kTpr) * V);
#pragma unroll
      for (int e = 0; e < V / 4; ++e) {
        const float4 w = __ldg(g + e);
        f[4 * e] = f[4 * e] * inv * w.x;
        f[4 * e + 1] = f[4 * e + 1] * inv * w.y;
        f[4 * e + 2] = f[4 * e + 2] * inv * w.z;
        f[4 * e + 3] = f[4 * e + 3] * inv * w.w;
      }
      if (!DP_DCHECK(in_buffer(row * d + static_cast<long long>(t + k * kTpr) * V, V, rows * d), 50u, nullptr)) continue;
      reinterpret_cast<uint4*>(Y + row * d)[t + k * kTpr] = pack16<T, V>(f, X);
    }
  }
}

// The warp's sums of a (in lanes 0 .. 15) and of b (in lanes 16 .. 31): the halves swap what they do
// not keep, so both take five exchanges.
__device__ __forceinline__ float half_sums(float a, float b, uint32_t lane) {
  const bool low = lane < 16;
  float x = (low ? a : b) + __shfl_xor_sync(0xFFFFFFFFu, low ? b : a, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

constexpr int kNormStagesMax = 8;

// Block (part, sample): rows [part per, part per + per) of the sample, one at a time, each held by
// all threads, NV vectors a thread.  Writes dh and the block's column sums of dy h r into
// parts[sample][part][d].  The rows of the tensors come through a ring of `stages` slots of shared
// memory, filled by bulk copies that thread 0 issues as soon as a slot's row is in registers: the
// copies of the next rows are in flight while this row is summed and written.  8 x 2048 rows of 4096 in
// bf16 with a residual gradient (537 MB): 89 us, 6.0 TB/s, with two blocks of 512 threads an SM.  Rows
// loaded straight to registers, 212 of them a thread, took 124 us; 256 threads with two vectors each, or
// three blocks an SM, 95 and 101.
template <typename T, int NV, bool RES>
__global__ void __launch_bounds__(512, NV == 1 ? 2 : 1)
    rmsnorm_backward_kernel(const T* __restrict__ H, const float* __restrict__ gain, const T* __restrict__ dY,
                            const T* __restrict__ dres, int T_len, int d, float eps, int per, int stages,
                            T* __restrict__ dX, float* __restrict__ parts, uint32_t* __restrict__ status) {
  constexpr int V = EmbVec<T>::N;
  constexpr int kTensors = RES ? 3 : 2;
  constexpr bool kGainHeld = NV < 4;  // else its values are read again for every row (from L1)
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kNormStagesMax];
  __shared__ float red[2][2][16];
  __shared__ int abort_word;
  const int t = threadIdx.x, threads = blockDim.x, warps = threads / 32;
  const uint32_t lane = lane_id();
  const int vecs = d / V;
  const uint32_t row_bytes = static_cast<uint32_t>(vecs) * 16u;
  const float inv_d = 1.0f / static_cast<float>(d);
  if (t == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_addr(full + s), 1);
    abort_word = 0;
    fence_mbar_init();
  }
  __syncthreads();
  griddep_enter();
  if (blockIdx.x == 0 && blockIdx.y == 0 && t == 0) *status = 0u;
  const int first = blockIdx.x * per;
  const int rows = min(per, T_len - first);
  const long long base = (static_cast<long long>(blockIdx.y) * T_len + first) * d;
  auto fetch = [&](int row, int slot) {  // thread 0
    const uint32_t bar = smem_addr(full + slot);
    const uint32_t dst = smem_addr(ring) + static_cast<uint32_t>(slot) * (kTensors * row_bytes);
    const long long at = base + static_cast<long long>(row) * d;
    mbar_arrive_expect_tx(bar, kTensors * row_bytes);
    bulk_load(dst, H + at, row_bytes, bar);
    bulk_load(dst + row_bytes, dY + at, row_bytes, bar);
    if constexpr (RES) bulk_load(dst + 2 * row_bytes, dres + at, row_bytes, bar);
  };
  if (t == 0)
    for (int s = 0; s < stages && s < rows; ++s) fetch(s, s);
  float g[kGainHeld ? NV : 1][V], acc[NV][V];
  auto gains = [&](int k, float (&out)[V]) {
    const float4* p = reinterpret_cast<const float4*>(gain + static_cast<long long>(t + k * threads) * V);
#pragma unroll
    for (int e = 0; e < V / 4; ++e) {
      const float4 w = __ldg(p + e);
      out[4 * e] = w.x;
      out[4 * e + 1] = w.y;
      out[4 * e + 2] = w.z;
      out[4 * e + 3] = w.w;
    }
  };
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int j = 0; j < V; ++j) acc[k][j] = 0.0f;
    if constexpr (kGainHeld) {
#pragma unroll
      for (int j = 0; j < V; ++j) g[k][j] = 0.0f;
      if (t + k * threads < vecs) gains(k, g[k]);
    }
  }
  int slot = 0, s = 0;
  uint32_t phase = 0;
  bool gave_up = false;
  for (; s < rows; ++s) {
    const bool ok = mbar_wait_bounded(smem_addr(full + slot), phase, &abort_word, status, 31u);
    const uint4* at = reinterpret_cast<const uint4*>(ring + static_cast<size_t>(slot) * (kTensors * row_bytes));
    uint4 qh[NV], qy[NV], qr[NV];
    float hh = 0.0f, uh = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = t + k * threads;
      qh[k] = qy[k] = qr[k] = make_uint4(0u, 0u, 0u, 0u);
      if (v < vecs) {
        qh[k] = at[v];
        qy[k] = at[vecs + v];
        if constexpr (RES) qr[k] = at[2 * vecs + v];
        float h[V], y[V], w[V];
        unpack16(qh[k], h, H);
        unpack16(qy[k], y, H);
        if constexpr (!kGainHeld) gains(k, w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          hh = fmaf(h[j], h[j], hh);
          uh = fmaf(y[j] * (kGainHeld ? g[kGainHeld ? k : 0][j] : w[j]), h[j], uh);
        }
      }
    }
    const int turn = s & 1;  // written again two rows on, after the barrier between
    const float half = half_sums(hh, uh, lane);
    if (lane % 16 == 0) red[turn][lane / 16][t / 32] = half;
    gave_up = __syncthreads_or(!ok);
    if (gave_up) break;  // a wait that ran out ends the block together
    if (t == 0 && s + stages < rows) fetch(s + stages, slot);
    float both = static_cast<int>(lane % 16) < warps ? red[turn][lane / 16][lane % 16] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) both += __shfl_xor_sync(0xFFFFFFFFu, both, o);
    hh = __shfl_sync(0xFFFFFFFFu, both, 0);
    uh = __shfl_sync(0xFFFFFFFFu, both, 16);
    const float inv = 1.0f / sqrtf(fmaf(hh, inv_d, eps));
    const float mean = inv * (uh * inv_d);  // of u_j h_j r: like u in size, where r^3 may be out of range
    const long long out_at = base + static_cast<long long>(s) * d;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = t + k * threads;
      if (v >= vecs) continue;
      float h[V], y[V], w[V], o[V];
      unpack16(qh[k], h, H);
      unpack16(qy[k], y, H);
      if constexpr (RES) unpack16(qr[k], o, H);
      if constexpr (!kGainHeld) gains(k, w);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float x = h[j] * inv;
        acc[k][j] = fmaf(y[j], x, acc[k][j]);
        const float dh = inv * fmaf(-x, mean, y[j] * (kGainHeld ? g[kGainHeld ? k : 0][j] : w[j]));
        o[j] = RES ? o[j] + dh : dh;
      }
      if (DP_DCHECK(first + s < T_len, 51u, status)) reinterpret_cast<uint4*>(dX + out_at)[v] = pack16<T, V>(o, H);
    }
    if (++slot == stages) {
      slot = 0;
      phase ^= 1u;
    }
  }
  if (gave_up) {  // no copy may still write the ring when the block leaves; this wait is bounded too
    if (t == 0) {
      const unsigned long long t0 = global_timer_ns();
      for (int k = 0; k < stages && s + k < rows; ++k) {
        const int at = slot + k < stages ? slot + k : slot + k - stages;
        const uint32_t parity = slot + k < stages ? phase : phase ^ 1u;
        while (!mbar_try_wait(smem_addr(full + at), parity) && global_timer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
    return;
  }
  float* out = parts + (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * d;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = t + k * threads;
    if (v >= vecs) continue;
#pragma unroll
    for (int e = 0; e < V / 4; ++e)
      reinterpret_cast<float4*>(out + static_cast<long long>(v) * V)[e] =
          make_float4(acc[k][4 * e], acc[k][4 * e + 1], acc[k][4 * e + 2], acc[k][4 * e + 3]);
  }
}

// per_sample[i][j] = sum over the sample's parts in fp64, blockIdx.y: sample.  Its 4 to 16 warps take the
// parts of 128 columns in turn, four columns a lane, and their sums are added in their order.  One thread a
// column, its parts in a row, made the step of 2048 rows of 768 (1024 parts) 58 us; this makes it 17 to 19.
constexpr int kPartsWarps = 16;  // at most
__global__ void __launch_bounds__(kPartsWarps * 32)
    rmsnorm_parts_kernel(const float* __restrict__ parts, int nparts, int d, float* __restrict__ per_sample) {
  griddep_enter();
  __shared__ double sums[kPartsWarps][128];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32, first = blockIdx.x * 128;
  const int j = first + 4 * lane;
  double v[4] = {0.0, 0.0, 0.0, 0.0};
  if (j < d) {
    const float* p = parts + static_cast<long long>(blockIdx.y) * nparts * d + j;
#pragma unroll 8
    for (int k = warp; k < nparts; k += warps) {
      const float4 x = *reinterpret_cast<const float4*>(p + static_cast<long long>(k) * d);
      v[0] += static_cast<double>(x.x);
      v[1] += static_cast<double>(x.y);
      v[2] += static_cast<double>(x.z);
      v[3] += static_cast<double>(x.w);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sums[warp][4 * lane + e] = v[e];
  __syncthreads();
  const int c = threadIdx.x;
  if (c >= 128 || first + c >= d) return;
  double sum = 0.0;
  for (int w = 0; w < warps; ++w) sum += sums[w][c];
  per_sample[static_cast<long long>(blockIdx.y) * d + first + c] = static_cast<float>(sum);
}

// The end of the backward in one launch, a cluster of 8 blocks that share the columns:
//   per_sample[i][j] = sum over the sample's parts, in part order;
//   norms[i] = ||per_sample[i]||, from the blocks' squares through distributed shared memory;
//   with S: S[j] = sum_i c_i per_sample[i][j] + std z_j.
// A thread holds four columns; threads left over take other samples beside them.  In place of two
// launches this takes 3.5 us off the shortest calls.  Eight SMs are too few for many parts (2 x 486 rows of
// 396, a part each: 65 us a step, 14 with the launch before), so those are summed by rmsnorm_parts_kernel first, and are then one part a sample (`parts`
// and `per_sample` are then the same array).
constexpr int kFinishCtas = 8;
constexpr int kFinishThreads = 512;
constexpr int kFinishChunk = 256;  // samples at a time
__global__ void __cluster_dims__(kFinishCtas, 1, 1) __launch_bounds__(kFinishThreads)
    rmsnorm_finish_kernel(const float* parts, int nparts, int B, int d, float* per_sample, float* __restrict__ norms,
                          float C, double noise_std, PhiloxKey key, uint32_t layer_id, StepRef step,
                          float* __restrict__ S) {
  griddep_enter();
  __shared__ float sq[kFinishChunk][kFinishThreads / 32];
  __shared__ float total[kFinishChunk];  // of this block's columns, read by the cluster
  __shared__ float c[kFinishChunk];
  __shared__ double lanes_s[kFinishThreads][4];
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_rank();
  const int quads = d / 4, per = (quads + kFinishCtas - 1) / kFinishCtas;
  const int first = static_cast<int>(rank) * per;
  const int mine = max(0, min(per, quads - first));
  const int width = min(kFinishThreads, (per + 31) / 32 * 32);  // threads a sample, whole warps (per <= 512)
  const int lanes = kFinishThreads / width, lane = tid / width, t = tid % width;
  const bool active = lane < lanes, has = active && t < mine;
  const long long col = 4ll * (first + t);
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  for (int base = 0; base < B; base += kFinishChunk) {
    const int count = min(kFinishChunk, B - base);
    if (active) {
      for (int s = lane; s < count; s += lanes) {
        float ss = 0.0f;
        if (has) {
          const float* p = parts + static_cast<long long>(base + s) * nparts * d + col;
          double v[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 8
          for (int k = 0; k < nparts; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(p + static_cast<long long>(k) * d);
            v[0] += static_cast<double>(x.x);
            v[1] += static_cast<double>(x.y);
            v[2] += static_cast<double>(x.z);
            v[3] += static_cast<double>(x.w);
          }
          const float4 f = make_float4(static_cast<float>(v[0]), static_cast<float>(v[1]), static_cast<float>(v[2]),
                                       static_cast<float>(v[3]));
          *reinterpret_cast<float4*>(per_sample + static_cast<long long>(base + s) * d + col) = f;
          ss = fmaf(f.x, f.x, fmaf(f.y, f.y, fmaf(f.z, f.z, f.w * f.w)));
        }
        ss = warp_sum(ss);
        if (t % 32 == 0) sq[s][t / 32] = ss;
      }
    }
    __syncthreads();
    for (int s = tid; s < count; s += kFinishThreads) {
      float sum = 0.0f;
      for (int w = 0; w < width / 32; ++w) sum += sq[s][w];
      total[s] = sum;
    }
    __syncwarp();
    cluster_sync_all();
    for (int s = tid; s < count; s += kFinishThreads) {
      double n2 = 0.0;
#pragma unroll
      for (uint32_t r = 0; r < kFinishCtas; ++r)
        n2 += static_cast<double>(__uint_as_float(ld_cluster_u32(smem_addr(&total[s]), r)));
      const float n = static_cast<float>(sqrt(n2));
      c[s] = clip_factor(n, C);
      if (rank == 0 && norms) norms[base + s] = n;
    }
    __syncthreads();
    if (S && has) {
#pragma unroll 4
      for (int s = lane; s < count; s += lanes) {  // the thread's own values again
        const float4 x = *reinterpret_cast<const float4*>(per_sample + static_cast<long long>(base + s) * d + col);
        const double w = static_cast<double>(c[s]);
        acc[0] = fma(w, static_cast<double>(x.x), acc[0]);
        acc[1] = fma(w, static_cast<double>(x.y), acc[1]);
        acc[2] = fma(w, static_cast<double>(x.z), acc[2]);
        acc[3] = fma(w, static_cast<double>(x.w), acc[3]);
      }
    }
    __syncwarp();
    cluster_sync_all();  // the totals were read: they may change, or the block may leave
  }
  if (!S) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) lanes_s[tid][e] = acc[e];
  __syncthreads();
  if (lane != 0 || !has) return;
  double z[4] = {0.0, 0.0, 0.0, 0.0};
  if (noise_std != 0.0)
    normals4(static_cast<uint32_t>(col / 4), layer_id, step.get(), kStreamNoise, key, z, NoiseTablesGlobal{}, noise_std);
  float o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    double sum = 0.0;
    for (int l = 0; l < lanes; ++l) sum += lanes_s[l * width + t][e];
    o[e] = static_cast<float>(sum + z[e]);
  }
  if (DP_DCHECK(col + 4 <= d, 52u, nullptr)) *reinterpret_cast<float4*>(S + col) = make_float4(o[0], o[1], o[2], o[3]);
}

// S[j] += sum_i c_i per_sample[i][j] for given norms, four columns a thread.
constexpr int kGainSamples = 1024;  // clip factors held at a time
constexpr int kGainSumThreads = 128;
__global__ void __launch_bounds__(kGainSumThreads)
    rmsnorm_sum_kernel(const float* __restrict__ per_sample, const float* __restrict__ norms, int B, int d, float C,
                       float* __restrict__ S) {
  griddep_enter();
  __shared__ float c[kGainSamples];
  __shared__ double acc_s[kGainSumThreads][4];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // 32 groups of 4 columns a block; the 4 warps share the samples, in a fixed split.
  const int j = (blockIdx.x * 32 + lane) * 4;
  double a[4] = {0.0, 0.0, 0.0, 0.0};
  for (int base = 0; base < B; base += kGainSamples) {
    const int count = min(kGainSamples, B - base);
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kGainSumThreads) c[i] = clip_factor(norms[base + i], C);
    __syncthreads();
    if (j < d) {
#pragma unroll 4
      for (int i = warp; i < count; i += kGainSumThreads / 32) {
        const float4 x = *reinterpret_cast<const float4*>(per_sample + static_cast<long long>(base + i) * d + j);
        const double w = static_cast<double>(c[i]);
        a[0] = fma(w, static_cast<double>(x.x), a[0]);
        a[1] = fma(w, static_cast<double>(x.y), a[1]);
        a[2] = fma(w, static_cast<double>(x.z), a[2]);
        a[3] = fma(w, static_cast<double>(x.w), a[3]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) acc_s[threadIdx.x][e] = a[e];
  __syncthreads();
  if (warp != 0 || j >= d) return;
  float4 o = *reinterpret_cast<const float4*>(S + j);
  float* of = &o.x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    double s = static_cast<double>(of[e]);
    for (int w = 0; w < kGainSumThreads / 32; ++w) s += acc_s[w * 32 + lane][e];
    of[e] = static_cast<float>(s);
  }
  if (DP_DCHECK(j + 4 <= d, 53u, nullptr)) *reinterpret_cast<float4*>(S + j) = o;
}

}  // namespace dpclip
