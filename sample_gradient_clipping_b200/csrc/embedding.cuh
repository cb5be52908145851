// The embedding table: its scaled lookup and its privatised gradient.
//
// The lookup is y_n = scale W[id_n].  Sample i's gradient of the table is sparse: row v of G_i is
// scale times the sum of the dY rows of the sample's tokens with id v, so
//   n_i^2 = scale^2 sum over groups (i, v) of || sum of the group's dY rows ||^2,
//   S[v]  = scale sum_i c_i (sum of group (i, v)) + sigma C z.
// As a linear layer it would be a one-hot X of V columns; here the tokens are sorted instead:
//   emb_sort_kernel  a stable radix sort of the tokens by id.  Token n = i T + t, so each id's run
//                    is ordered by sample and each group is contiguous; the kernel also lists the
//                    groups and the rows that occur.
//   emb_norm_kernel  the sum of every group, squared, into a slot of the group's first token; the
//                    sum of a long group is kept in fp32, since the last kernel needs it again.
//   emb_norms_kernel n_i from the sample's slots, in a fixed order in fp64.
//   emb_sum_kernel   every row of S: its groups times their clip factors, plus the noise.
// dY is read twice (the norm decides the factor of every row before any row can be added), S is
// written once.  Nothing is added with floating-point atomics, so the bits repeat.
// A token whose id is negative, at or past V, or the padding index belongs to no group; an id at
// or past V is also recorded in the status word.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "rng.cuh"
#include "simt.cuh"
#include "umma_gemm_2sm.cuh"

namespace dpclip {

// Status word of an id at or past V (a timeout's site is below it, a debug check's above).
constexpr uint32_t kStatusIdRange = 900u;

constexpr int kEmbSortCtas = 8;       // one cluster: its barriers are the passes' barriers
constexpr int kEmbSortThreads = 1024;
constexpr int kEmbRadix = 256;
// A group of more tokens than this is summed by a whole block, and its sum kept: the last kernel
// then reads 4 bytes an element once instead of its rows (2 bytes each in bf16).
constexpr int kEmbLongGroup = 16;
// A row of S with more tokens than this is formed by a whole block.
constexpr int kEmbHeavyRow = 64;
constexpr int kEmbThreads = 256;
constexpr int kEmbWarps = kEmbThreads / 32;

enum EmbCount : int { kEmbGroups = 0, kEmbLong = 1, kEmbHeavy = 2 };

// The sorted tokens of one call (all device pointers into the workspace).
struct EmbIndex {
  uint32_t* keys[2];     // [N] ids, ping-pong between the passes
  uint32_t* toks[2];     // [N] tokens
  int last;              // which of the two holds the sorted order
  uint32_t* counts;      // EmbCount
  uint32_t* row_first;   // [V] 1 + first group of the row, 0: the row does not occur
  uint32_t* row_end;     // [V] one past its last group (rows that occur)
  uint32_t* group_pos;   // [groups + 1] first sorted position of the group
  int* group_long;       // [groups] slot of a long group's sum, or -1
  uint32_t* long_list;   // groups by slot
  uint32_t* heavy_list;  // rows
  float* sq;             // [N][chunks] squared sums, by first token of the group
  float* long_sums;      // [slots][d]
};

template <typename T>
struct EmbVec;  // 16 bytes of a dY row as fp32
template <>
struct EmbVec<__nv_bfloat16> {
  static constexpr int N = 8;
};
template <>
struct EmbVec<float> {
  static constexpr int N = 4;
};

__device__ __forceinline__ void unpack16(const uint4& q, float (&f)[8], const __nv_bfloat16*) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack16(const uint4& q, float (&f)[4], const float*) {
  f[0] = __uint_as_float(q.x);
  f[1] = __uint_as_float(q.y);
  f[2] = __uint_as_float(q.z);
  f[3] = __uint_as_float(q.w);
}

// ------------------------------------------------------------------------------------ lookup
// y[n, :] = scale W[id_n, :], VEC elements per thread and step; ids outside [0, V) give zeros.
// Bound by HBM: it reads a table row and writes an output row per token.
template <typename TI, typename TO, int VEC>
__global__ void emb_lookup_kernel(const TI* __restrict__ W, const void* __restrict__ ids, int index64, float scale,
                                  long long N, int V, int d, TO* __restrict__ Y) {
  griddep_enter();
  const int per_row = d / VEC;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  const long long first = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  // (row, col) of the thread's vector moves by a fixed step, so nothing is divided in the loop.
  const long long step_row = stride / per_row;
  const int step_col = static_cast<int>(stride % per_row);
  long long row = first / per_row;
  int col = static_cast<int>(first % per_row);
  constexpr int kU = 4;  // vectors in flight per thread
  while (row < N) {
    float f[kU][VEC];
    long long out[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      out[u] = -1;
      if (row >= N) continue;
      const long long id = index64 ? static_cast<const long long*>(ids)[row] : static_cast<const int*>(ids)[row];
      out[u] = row * d + static_cast<long long>(col) * VEC;
      if (id >= 0 && id < V) {
        const TI* src = W + id * d + static_cast<long long>(col) * VEC;
        constexpr int kPer = EmbVec<TI>::N;
#pragma unroll
        for (int q = 0; q < VEC / kPer; ++q) {
          float g[kPer];
          unpack16(__ldg(reinterpret_cast<const uint4*>(src) + q), g, src);
#pragma unroll
          for (int e = 0; e < kPer; ++e) f[u][q * kPer + e] = g[e] * scale;
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[u][e] = 0.0f;
      }
      row += step_row;
      col += step_col;
      if (col >= per_row) {
        col -= per_row;
        ++row;
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (out[u] < 0) continue;
      if (!DP_DCHECK(in_buffer(out[u], VEC, N * d), 40u, nullptr)) continue;
      if constexpr (sizeof(TO) == 2) {
        uint4 pk;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&pk);
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) h[e] = __floats2bfloat162_rn(f[u][2 * e], f[u][2 * e + 1]);
        *reinterpret_cast<uint4*>(Y + out[u]) = pk;
      } else {
#pragma unroll
        for (int q = 0; q < VEC / 4; ++q)
          *reinterpret_cast<float4*>(Y + out[u] + 4 * q) =
              make_float4(f[u][4 * q], f[u][4 * q + 1], f[u][4 * q + 2], f[u][4 * q + 3]);
      }
    }
  }
}

// -------------------------------------------------------------------------------------- sort
// Shared-memory word of CTA `rank`'s copy of the variable at `local`.
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t local, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(local, rank)) : "memory");
  return v;
}

// The cluster's barrier, after the threads of each warp have met again.
__device__ __forceinline__ void emb_cluster_sync() {
  __syncwarp();
  cluster_sync_all();
}

// The id of token n as a sort key: V for a token that belongs to no group.
__device__ __forceinline__ uint32_t emb_key(const void* ids, int index64, long long n, int V, long long padding,
                                            uint32_t* status) {
  const long long id = index64 ? static_cast<const long long*>(ids)[n] : static_cast<const int*>(ids)[n];
  if (id >= V) *status = kStatusIdRange;
  return (id < 0 || id >= V || id == padding) ? static_cast<uint32_t>(V) : static_cast<uint32_t>(id);
}

// Sorts the N tokens by key in `passes` stable passes of 8 bits, then lists the groups.  One
// cluster of 8 blocks: token ranges are contiguous per block and per warp, so a warp's rank within
// a digit is (digits below) + (blocks before) + (warps before) + (its own so far), and the only
// exchange is each block's 256 digit totals through distributed shared memory.  All the work is
// latency (a few microseconds a pass at 16384 tokens), which one launch keeps smallest.
__global__ void __cluster_dims__(kEmbSortCtas, 1, 1) __launch_bounds__(kEmbSortThreads, 1)
    emb_sort_kernel(const void* __restrict__ ids, int index64, long long N, int T, int V, long long padding,
                    int passes, EmbIndex ix, long long sq_len, uint32_t* __restrict__ status) {
  griddep_enter();
  constexpr int kWarps = kEmbSortThreads / 32;
  __shared__ uint32_t hist[kWarps][kEmbRadix];  // counts, then each warp's next position per digit
  __shared__ uint32_t total[kEmbRadix];         // this block's digit totals, read by the cluster
  __shared__ uint32_t scan[kEmbRadix];
  __shared__ uint32_t heads[2];                 // group heads in this block
  __shared__ uint32_t warp_heads[kWarps];
  const int tid = threadIdx.x, warp = tid / 32;
  const uint32_t lane = lane_id();
  const uint32_t rank = cluster_rank();
  const int gthread = static_cast<int>(rank) * kEmbSortThreads + tid;
  constexpr int kAll = kEmbSortCtas * kEmbSortThreads;

  for (long long v = gthread; v < V; v += kAll) ix.row_first[v] = 0u;
  for (long long k = gthread; k < sq_len; k += kAll) ix.sq[k] = 0.0f;
  if (gthread == 0) {
    *status = 0u;
    ix.counts[kEmbLong] = 0u;
    ix.counts[kEmbHeavy] = 0u;
  }
  emb_cluster_sync();  // the status word is cleared before a key may set it

  // Every warp owns one contiguous range of positions, in (block, warp) order.
  const long long per = ((N + kEmbSortCtas * kWarps - 1) / (kEmbSortCtas * kWarps) + 31) / 32 * 32;
  const long long w0 = (static_cast<long long>(rank) * kWarps + warp) * per;
  const long long begin = w0 < N ? w0 : N;
  const long long end = begin + per < N ? begin + per : N;
  const uint32_t below = (1u << lane) - 1u;

  for (int pass = 0; pass < passes; ++pass) {
    const int shift = 8 * pass;
    const uint32_t* kin = ix.keys[(pass + 1) & 1];
    const uint32_t* tin = ix.toks[(pass + 1) & 1];
    uint32_t* kout = ix.keys[pass & 1];
    uint32_t* tout = ix.toks[pass & 1];
    for (int q = tid; q < kWarps * kEmbRadix; q += kEmbSortThreads) (&hist[0][0])[q] = 0u;
    __syncthreads();
    for (long long p = begin + lane; p < end; p += 32) {
      const uint32_t key = pass ? __ldcg(kin + p) : emb_key(ids, index64, p, V, padding, status);
      atomicAdd(&hist[warp][(key >> shift) & (kEmbRadix - 1)], 1u);
    }
    __syncthreads();
    if (tid < kEmbRadix) {
      uint32_t sum = 0;
#pragma unroll 8
      for (int w = 0; w < kWarps; ++w) {
        const uint32_t c = hist[w][tid];
        hist[w][tid] = sum;
        sum += c;
      }
      total[tid] = sum;
    }
    emb_cluster_sync();
    uint32_t before = 0, all = 0;
    if (tid < kEmbRadix) {
#pragma unroll
      for (uint32_t r = 0; r < kEmbSortCtas; ++r) {
        const uint32_t c = ld_cluster_u32(smem_addr(&total[tid]), r);
        all += c;
        if (r < rank) before += c;
      }
      scan[tid] = all;
    }
    __syncthreads();
    // Exclusive sum of the 256 digit totals by warp 0, 8 digits a lane.
    if (warp == 0) {
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = sum;
        sum += scan[8 * lane + e];
      }
      uint32_t run = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, run, o);
        if (lane >= static_cast<uint32_t>(o)) run += x;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) scan[8 * lane + e] = run - sum + c[e];
    }
    __syncthreads();
    if (tid < kEmbRadix) {
      const uint32_t base = scan[tid] + before;
#pragma unroll 8
      for (int w = 0; w < kWarps; ++w) hist[w][tid] += base;
    }
    __syncthreads();
    for (long long p0 = begin; p0 < end; p0 += 32) {
      const long long p = p0 + lane;
      const bool ok = p < end;
      const uint32_t key = !ok ? 0u : pass ? __ldcg(kin + p) : emb_key(ids, index64, p, V, padding, status);
      const uint32_t tok = !ok ? 0u : pass ? __ldcg(tin + p) : static_cast<uint32_t>(p);
      const uint32_t digit = ok ? (key >> shift) & (kEmbRadix - 1) : kEmbRadix;  // a lane without a token: no digit
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, digit);
      uint32_t pos = 0;
      if (ok) pos = hist[warp][digit] + __popc(same & below);
      __syncwarp();
      if (ok && (same & below) == 0u) hist[warp][digit] += __popc(same);
      __syncwarp();
      if (ok && DP_DCHECK(static_cast<long long>(pos) < N, 41u, status)) {
        __stcg(kout + pos, key);
        __stcg(tout + pos, tok);
      }
    }
    emb_cluster_sync();  // the pass's arrays are whole, and `total` is free
  }

  // Group heads: a position whose id or sample differs from the one before.  Position N counts as
  // a token of no group, so the first such position closes the last group.
  const uint32_t* keys = ix.keys[ix.last];
  const uint32_t* toks = ix.toks[ix.last];
  const uint32_t none = static_cast<uint32_t>(V);
  auto head = [&](long long p, bool& close) {
    const uint32_t key = p < N ? __ldcg(keys + p) : none;
    const uint32_t prev = p > 0 ? __ldcg(keys + p - 1) : none;
    close = key == none && (p == 0 || prev != none);
    if (key == none) return false;
    return p == 0 || prev != key || __ldcg(toks + p - 1) / static_cast<uint32_t>(T) != __ldcg(toks + p) / static_cast<uint32_t>(T);
  };
  // The warp of the last token also takes position N.
  const long long hend = (begin < N && end == N) ? N + 1 : end;
  uint32_t mine = 0;
  for (long long p0 = begin; p0 < hend; p0 += 32) {
    bool close = false;
    const bool h = p0 + lane < hend && head(p0 + lane, close);
    mine += __popc(__ballot_sync(0xFFFFFFFFu, h));
  }
  if (lane == 0) warp_heads[warp] = mine;
  __syncthreads();
  if (tid == 0) {
    uint32_t sum = 0;
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t c = warp_heads[w];
      warp_heads[w] = sum;
      sum += c;
    }
    heads[0] = sum;
  }
  emb_cluster_sync();
  if (tid == 0) {
    uint32_t base = 0, all = 0;
    for (uint32_t r = 0; r < kEmbSortCtas; ++r) {
      const uint32_t c = ld_cluster_u32(smem_addr(&heads[0]), r);
      all += c;
      if (r < rank) base += c;
    }
    heads[1] = base;
    if (rank == 0) ix.counts[kEmbGroups] = all;
  }
  __syncthreads();
  uint32_t next = heads[1] + warp_heads[warp];
  for (long long p0 = begin; p0 < hend; p0 += 32) {
    bool close = false;
    const bool h = p0 + lane < hend && head(p0 + lane, close);
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, h);
    const uint32_t g = next + __popc(mask & below);
    if ((h || close) && DP_DCHECK(static_cast<long long>(g) <= N, 42u, status))
      __stcg(ix.group_pos + g, static_cast<uint32_t>(p0 + lane));
    next += __popc(mask);
  }
  emb_cluster_sync();
  const uint32_t groups = __ldcg(ix.counts + kEmbGroups);
  for (uint32_t g = gthread; g < groups; g += kAll) {
    const uint32_t p = __ldcg(ix.group_pos + g), q = __ldcg(ix.group_pos + g + 1);
    const uint32_t key = __ldcg(keys + p);
    int slot = -1;
    if (q - p > kEmbLongGroup) {
      slot = static_cast<int>(atomicAdd(ix.counts + kEmbLong, 1u));
      ix.long_list[slot] = g;
    }
    ix.group_long[g] = slot;
    if (p == 0 || __ldcg(keys + p - 1) != key) {
      ix.row_first[key] = g + 1;
      const long long far = static_cast<long long>(p) + kEmbHeavyRow;
      if (far < N && __ldcg(keys + far) == key) ix.heavy_list[atomicAdd(ix.counts + kEmbHeavy, 1u)] = key;
    }
    if (q >= N || __ldcg(keys + q) != key) ix.row_end[key] = g + 1;
  }
}

// ------------------------------------------------------------------------------------- norms
// Adds the dY rows of sorted positions p, p + step, .. below `end` to acc (this lane's vector of
// the chunk).  The tokens of 32 rows are fetched by one load, and kU rows are in flight.
template <typename T>
__device__ __forceinline__ void emb_add_rows(const T* __restrict__ dY, const uint32_t* __restrict__ toks,
                                             uint32_t p, uint32_t step, uint32_t end, int d, int col, bool col_ok,
                                             uint32_t lane, float (&acc)[EmbVec<T>::N]) {
  constexpr int V = EmbVec<T>::N;
  constexpr int kU = 8;
  for (uint32_t base = p; base < end; base += 32 * step) {
    const uint32_t at = base + lane * step;
    const uint32_t tok = at < end ? toks[at] : 0u;
    const int rows = static_cast<int>(min((end - base + step - 1) / step, 32u));
    for (int k0 = 0; k0 < rows; k0 += kU) {
      uint4 q[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t t = __shfl_sync(0xFFFFFFFFu, tok, (k0 + u) & 31);
        q[u] = make_uint4(0u, 0u, 0u, 0u);
        if (k0 + u < rows && col_ok) q[u] = __ldg(reinterpret_cast<const uint4*>(dY + static_cast<long long>(t) * d + col));
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (k0 + u < rows) {
          float f[V];
          unpack16(q[u], f, dY);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] += f[e];
        }
      }
    }
  }
}

// blockIdx.y: chunk of 32 vectors of 16 bytes.  Long groups first, each by a block whose warps
// share its rows; then one group per warp.
template <typename T>
__global__ void __launch_bounds__(kEmbThreads) emb_norm_kernel(const T* __restrict__ dY, int d, EmbIndex ix) {
  griddep_enter();
  constexpr int V = EmbVec<T>::N;
  __shared__ float part[kEmbWarps][32 * V];
  const int warp = threadIdx.x / 32;
  const uint32_t lane = lane_id();
  const int chunk = blockIdx.y, chunks = gridDim.y;
  const int col = chunk * 32 * V + static_cast<int>(lane) * V;
  const bool col_ok = col < d;
  const uint32_t* toks = ix.toks[ix.last];
  const uint32_t groups = ix.counts[kEmbGroups], longs = ix.counts[kEmbLong];
  for (uint32_t slot = blockIdx.x; slot < longs; slot += gridDim.x) {
    const uint32_t g = ix.long_list[slot];
    const uint32_t p = ix.group_pos[g], q = ix.group_pos[g + 1];
    float acc[V] = {};
    emb_add_rows(dY, toks, p + warp, kEmbWarps, q, d, col, col_ok, lane, acc);
#pragma unroll
    for (int e = 0; e < V; ++e) part[warp][e * 32 + lane] = acc[e];
    __syncthreads();
    if (warp == 0) {
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kEmbWarps; ++w) s += part[w][e * 32 + lane];
        acc[e] = s;
        ss = fmaf(s, s, ss);
      }
      if (col_ok) {
        float4* out = reinterpret_cast<float4*>(ix.long_sums + static_cast<long long>(slot) * d + col);
#pragma unroll
        for (int e = 0; e < V / 4; ++e) out[e] = make_float4(acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]);
      }
      ss = warp_sum(ss);
      if (lane == 0) ix.sq[static_cast<long long>(toks[p]) * chunks + chunk] = ss;
    }
    __syncthreads();
  }
  for (uint32_t g = blockIdx.x * kEmbWarps + warp; g < groups; g += gridDim.x * kEmbWarps) {
    const uint32_t p = ix.group_pos[g], q = ix.group_pos[g + 1];
    if (q - p > kEmbLongGroup) continue;
    float acc[V] = {};
    emb_add_rows(dY, toks, p, 1u, q, d, col, col_ok, lane, acc);
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < V; ++e) ss = fmaf(acc[e], acc[e], ss);
    ss = warp_sum(ss);
    if (lane == 0) ix.sq[static_cast<long long>(toks[p]) * chunks + chunk] = ss;
  }
}

// norms[i] = |scale| sqrt(sum of the sample's T * chunks slots): one block a sample, fp64, in a
// fixed order.
__global__ void emb_norms_kernel(const float* __restrict__ sq, long long per_sample, float scale,
                                 float* __restrict__ norms, float* __restrict__ norms_out) {
  griddep_enter();
  __shared__ double part[kEmbWarps];
  const float* mine = sq + static_cast<long long>(blockIdx.x) * per_sample;
  double acc = 0.0;
  for (long long k = threadIdx.x; k < per_sample; k += kEmbThreads) acc += static_cast<double>(mine[k]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kEmbWarps; ++w) s += part[w];
    const float n = static_cast<float>(fabs(static_cast<double>(scale)) * sqrt(s));
    if (norms) norms[blockIdx.x] = n;
    if (norms_out) norms_out[blockIdx.x] = n;
  }
}

// --------------------------------------------------------------------------------------- sum
// acc += sum over groups first, first + step, .. below `end` of scale c_i (group's sum).
template <typename T>
__device__ __forceinline__ void emb_add_groups(const T* __restrict__ dY, const EmbIndex& ix, uint32_t first,
                                               uint32_t step, uint32_t end, int T_len, const float* __restrict__ norms,
                                               float C, float scale, int d, int col, bool col_ok, uint32_t lane,
                                               float (&acc)[EmbVec<T>::N]) {
  constexpr int V = EmbVec<T>::N;
  const uint32_t* toks = ix.toks[ix.last];
  for (uint32_t g = first; g < end; g += step) {
    const uint32_t p = ix.group_pos[g], q = ix.group_pos[g + 1];
    const int slot = ix.group_long[g];
    const float w = scale * clip_factor(norms[toks[p] / static_cast<uint32_t>(T_len)], C);
    float s[V] = {};
    if (slot >= 0) {
      if (col_ok) {
        const float4* in = reinterpret_cast<const float4*>(ix.long_sums + static_cast<long long>(slot) * d + col);
#pragma unroll
        for (int e = 0; e < V / 4; ++e) {
          const float4 x = in[e];
          s[4 * e] = x.x;
          s[4 * e + 1] = x.y;
          s[4 * e + 2] = x.z;
          s[4 * e + 3] = x.w;
        }
      }
    } else {
      emb_add_rows(dY, toks, p, 1u, q, d, col, col_ok, lane, s);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = fmaf(w, s[e], acc[e]);
  }
}

// S[v, :] (+)= its groups' clipped sums + std z, blockIdx.y: chunk as above.  Heavy rows first,
// each by a block; then one row per warp.  ACCUMULATE: rows that occur are added to, the others
// left alone.  NOISE: Box-Muller tables in shared memory; the normals' fp64 arithmetic is then what
// bounds the kernel (2 fp64 pipes' worth a pair), the stores otherwise.
template <typename T, bool NOISE, bool ACCUMULATE>
__global__ void __launch_bounds__(kEmbThreads)
    emb_sum_kernel(const T* __restrict__ dY, EmbIndex ix, int T_len, int V_rows, int d, const float* __restrict__ norms,
                   float C, float scale, double noise_std, PhiloxKey key, uint32_t layer_id, StepRef step,
                   float* __restrict__ S) {
  griddep_enter();
  constexpr int V = EmbVec<T>::N;
  __shared__ float part[kEmbWarps][32 * V];
  __shared__ double2 tab_s[NOISE ? kNoiseSharedEntries : 1];
  if constexpr (NOISE) stage_noise_tables(tab_s);
  __syncthreads();
  const uint32_t step_lo = NOISE ? step.get() : 0u;
  const int warp = threadIdx.x / 32;
  const uint32_t lane = lane_id();
  const int col = blockIdx.y * 32 * V + static_cast<int>(lane) * V;
  const bool col_ok = col < d;
  auto store = [&](long long v, float (&acc)[V]) {
    if (!col_ok || !DP_DCHECK(in_buffer(v * d + col, V, static_cast<long long>(V_rows) * d), 43u, nullptr)) return;
    float4* out = reinterpret_cast<float4*>(S + v * d + col);
#pragma unroll
    for (int e = 0; e < V / 4; ++e) {
      float4 x = make_float4(acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]);
      if constexpr (NOISE) {
        double z[4];
        normals4(static_cast<uint32_t>((static_cast<unsigned long long>(v) * d + col) / 4 + e), layer_id, step_lo,
                 kStreamNoise, key, z, NoiseTablesShared{tab_s}, noise_std);
        x.x = static_cast<float>(static_cast<double>(x.x) + z[0]);
        x.y = static_cast<float>(static_cast<double>(x.y) + z[1]);
        x.z = static_cast<float>(static_cast<double>(x.z) + z[2]);
        x.w = static_cast<float>(static_cast<double>(x.w) + z[3]);
      }
      if constexpr (ACCUMULATE) {
        const float4 o = out[e];
        x = make_float4(o.x + x.x, o.y + x.y, o.z + x.z, o.w + x.w);
      }
      out[e] = x;
    }
  };
  const uint32_t heavy = ix.counts[kEmbHeavy];
  for (uint32_t h = blockIdx.x; h < heavy; h += gridDim.x) {
    const uint32_t v = ix.heavy_list[h];
    const uint32_t first = ix.row_first[v] - 1, end = ix.row_end[v];
    float acc[V] = {};
    emb_add_groups(dY, ix, first + warp, kEmbWarps, end, T_len, norms, C, scale, d, col, col_ok, lane, acc);
#pragma unroll
    for (int e = 0; e < V; ++e) part[warp][e * 32 + lane] = acc[e];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kEmbWarps; ++w) s += part[w][e * 32 + lane];
        acc[e] = s;
      }
      store(v, acc);
    }
    __syncthreads();
  }
  for (long long v = static_cast<long long>(blockIdx.x) * kEmbWarps + warp; v < V_rows;
       v += static_cast<long long>(gridDim.x) * kEmbWarps) {
    const uint32_t first = ix.row_first[v];
    float acc[V] = {};
    if (first) {
      const uint32_t end = ix.row_end[v];
      if (ix.group_pos[end] - ix.group_pos[first - 1] > kEmbHeavyRow) continue;
      emb_add_groups(dY, ix, first - 1, 1u, end, T_len, norms, C, scale, d, col, col_ok, lane, acc);
    } else if (ACCUMULATE) {
      continue;
    }
    store(v, acc);
  }
}

}  // namespace dpclip
