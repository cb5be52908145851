// The embedding table: its scaled lookup and its privatised gradient.
//
// The lookup is y_n = scale W[id_n].  Sample i's gradient of the table is sparse: row v of G_i is
// scale times the sum of the dY rows of the sample's tokens with id v, so
//   n_i^2 = scale^2 sum over groups (i, v) of || sum of the group's dY rows ||^2,
//   S[v]  = scale sum_i c_i (sum of group (i, v)) + sigma C z.
// As a linear layer it would be a one-hot X of V columns; here the tokens are sorted instead:
//   emb_sort_kernel  a stable radix sort of the tokens by id.  Token n = i T + t, so each id's run
//                    is ordered by sample, and each group is contiguous;
//   emb_mark_kernel  finds the groups and rows in that order (a small sort does so itself);
//   emb_norm_kernel  puts the square of each group's sum into the slot of its first token; the sum
//                    of a long group is kept in fp32, since the last kernel needs it again;
//   emb_norms_kernel n_i from the sample's slots, in a fixed order in fp64;
//   emb_sum_kernel   every row of S: its tokens' rows (or its long groups' sums) times their clip
//                    factors, plus the noise.
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

constexpr int kEmbSortThreads = 1024;
constexpr int kEmbSortWarps = kEmbSortThreads / 32;
// A group of more tokens than this is summed by a whole block, and its sum kept: the last kernel
// then reads 4 bytes an element once instead of its rows (2 bytes each in bf16).
constexpr int kEmbLongGroup = 16;
// A row of S with more tokens than this is formed by a whole block.
constexpr int kEmbHeavyRow = 64;
constexpr int kEmbThreads = 256;
constexpr int kEmbWarps = kEmbThreads / 32;

// What the last kernel does at a sorted position: add the token's row; nothing, inside a long
// group; add the long group's sum, at its first position.
enum EmbUse : uint8_t { kEmbRow = 0, kEmbSkip = 1, kEmbLongSum = 2, kEmbUseMask = 3 };
constexpr uint8_t kEmbHead = 4;  // beside it: a group starts here (or the tokens without one do)

// The slot of a long group's sum: two groups of more than kEmbLongGroup tokens start at least
// that many + 1 positions apart.
__host__ __device__ constexpr long long emb_slot(long long first) { return first / (kEmbLongGroup + 1); }

// The sorted tokens of one call (device pointers into the workspace).
struct EmbIndex {
  const uint32_t* keys;  // [N] ids in order, V for a token without a group
  const uint32_t* toks;  // [N] their tokens
  uint32_t* heavies;     // how many heavy rows are listed
  uint32_t* heavy_list;  // their ids
  uint32_t* longs;       // how many long groups are listed
  uint2* long_list;      // their (first, end) positions
  uint2* rows;           // [V] (1 + first position, end position); (0, -): the row does not occur
  uint8_t* use;          // [N] EmbUse | kEmbHead
  uint32_t* turns;       // [chunks of emb_sum_kernel] rows handed out
  float* sq;             // [N][chunks] squared sums, by first token of the group; 0 elsewhere
  int chunks;            // of emb_norm_kernel
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

// The same for wide rows: blockIdx.y is a segment of 128 vectors, a warp takes one row's segment at a
// time, four vectors a lane, so the id is read once for 128 vectors and no place is computed twice.
// 16384 tokens of 4096 in bf16: 39 us for uniform ids (268 MB, 6.9 TB/s; the table's rows partly stay in
// L2), 31 us for ids as frequent as 1 / rank, against 58 and 50 us in the form above.
template <typename TI, typename TO>
__global__ void __launch_bounds__(256)
    emb_lookup_wide_kernel(const TI* __restrict__ W, const void* __restrict__ ids, int index64, float scale, long long N,
                           int V, int d, TO* __restrict__ Y) {
  griddep_enter();
  constexpr int kIn = EmbVec<TI>::N;  // elements of a 16-byte load; a thread's vector is 8 elements
  const int lane = static_cast<int>(lane_id());
  const int col0 = (blockIdx.y * 128 + lane) * 8;
  const long long stride = static_cast<long long>(gridDim.x) * 8;
  for (long long row = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32; row < N; row += stride) {
    const long long id = index64 ? static_cast<const long long*>(ids)[row] : static_cast<const int*>(ids)[row];
    const bool in = id >= 0 && id < V;
    const TI* src = W + (in ? id : 0) * d;
    uint4 q[4][8 / kIn];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < 8 / kIn; ++e) {
        q[u][e] = make_uint4(0u, 0u, 0u, 0u);
        if (in && col0 + 256 * u < d) q[u][e] = __ldg(reinterpret_cast<const uint4*>(src + col0 + 256 * u) + e);
      }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int col = col0 + 256 * u;
      if (col >= d || !DP_DCHECK(in_buffer(row * d + col, 8, N * d), 44u, nullptr)) continue;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8 / kIn; ++e) {
        float g[kIn];
        unpack16(q[u][e], g, src);
#pragma unroll
        for (int k = 0; k < kIn; ++k) f[e * kIn + k] = g[k] * scale;
      }
      TO* out = Y + row * d + col;
      if constexpr (sizeof(TO) == 2) {
        uint4 pk;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&pk);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
        *reinterpret_cast<uint4*>(out) = pk;
      } else {
        reinterpret_cast<float4*>(out)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(out)[1] = make_float4(f[4], f[5], f[6], f[7]);
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

// The id of token n as a sort key: V for a token that belongs to no group.
__device__ __forceinline__ uint32_t emb_key(const void* ids, int index64, long long n, int V, long long padding,
                                            uint32_t* status) {
  const long long id = index64 ? static_cast<const long long*>(ids)[n] : static_cast<const int*>(ids)[n];
  if (id >= V) *status = kStatusIdRange;
  return (id < 0 || id >= V || id == padding) ? static_cast<uint32_t>(V) : static_cast<uint32_t>(id);
}

// The end of the group of (key, sample) that starts at sorted position `first`, at most T positions
// on: a 32-way search by one warp.
__device__ __forceinline__ uint32_t emb_group_end(const EmbIndex& ix, uint32_t key, uint32_t sample, long long first,
                                                  long long N, uint32_t T, uint32_t lane) {
  long long lo = first, hi = first + T < N ? first + T : N;  // lo is inside, hi is not
  while (hi - lo > 1) {
    const long long step = (hi - lo + 31) / 32;
    const long long at = lo + step * (lane + 1);
    const bool inside = at < hi && __ldcg(ix.keys + at) == key && __ldcg(ix.toks + at) / T == sample;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, inside));
    const long long next = lo + step * (n + 1);
    hi = next < hi ? next : hi;
    lo += step * n;
  }
  return static_cast<uint32_t>(hi);
}

// Marks 32 sorted positions from p0: which start a group or a row, which lie in a long group, what
// the norm kernel's slots start from.  A long group is seen from the heads of three windows of 32:
// if none lies within 32 positions on one side, the group is long.  One warp.
__device__ __forceinline__ void emb_mark(const EmbIndex& ix, long long p0, long long N, uint32_t T, uint32_t none,
                                         uint32_t lane) {
  // The heads of a window, and this lane's key and token in the middle one.
  uint32_t my_key = none, my_tok = 0;
  bool my_row_head = false;
  auto heads = [&](long long w0, bool mine) {
    const long long p = w0 + lane;
    bool head = p >= N;  // the end closes the last group
    if (p >= 0 && p < N) {
      const uint32_t key = __ldcg(ix.keys + p), tok = __ldcg(ix.toks + p);
      const uint32_t last_key = p > 0 ? __ldcg(ix.keys + p - 1) : none + 1u, last_tok = p > 0 ? __ldcg(ix.toks + p - 1) : 0u;
      const bool row_head = key != last_key;
      head = row_head || (key != none && tok / T != last_tok / T);
      if (mine) {
        my_key = key;
        my_tok = tok;
        my_row_head = row_head;
      }
    }
    return __ballot_sync(0xFFFFFFFFu, head);
  };
  const uint32_t before = heads(p0 - 32, false), here = heads(p0, true), after = heads(p0 + 32, false);
  const uint32_t row_heads = __ballot_sync(0xFFFFFFFFu, my_row_head || p0 + lane >= N);
  const long long p = p0 + lane;
  const uint32_t upto = 0xFFFFFFFFu >> (31u - lane), past = ~upto;
  // First and end position of the group, relative to p0; "far" where no head is in sight.
  const bool head = (here >> lane) & 1u;
  const int first = (here & upto) ? 31 - __clz(here & upto) : before ? -1 - __clz(before) : -1000;
  const int end = (here & past) ? __ffs(here & past) - 1 : after ? 31 + __ffs(after) : 1000;
  const bool token = p < N && my_key < none;
  const bool is_long = token && end - first > kEmbLongGroup;
  // The long groups that start here, one by one by the whole warp.
  uint32_t starts = __ballot_sync(0xFFFFFFFFu, is_long && head);
  while (starts) {
    const int k = __ffs(starts) - 1;
    starts &= starts - 1u;
    const uint32_t stop = emb_group_end(ix, __shfl_sync(0xFFFFFFFFu, my_key, k), __shfl_sync(0xFFFFFFFFu, my_tok, k) / T,
                                        p0 + k, N, T, lane);
    if (lane == 0) ix.long_list[atomicAdd(ix.longs, 1u)] = make_uint2(static_cast<uint32_t>(p0) + k, stop);
  }
  if (p >= N) return;
  ix.use[p] = (is_long ? (head ? kEmbLongSum : kEmbSkip) : kEmbRow) | (head ? kEmbHead : 0);
  for (int c = 0; c < ix.chunks; ++c) ix.sq[static_cast<long long>(my_tok) * ix.chunks + c] = 0.0f;
  if (!token) return;
  if (my_row_head) {
    ix.rows[my_key].x = static_cast<uint32_t>(p) + 1u;
    const long long h = p + kEmbHeavyRow;
    if (h < N && __ldcg(ix.keys + h) == my_key) ix.heavy_list[atomicAdd(ix.heavies, 1u)] = my_key;
  }
  // The row ends here if the next position is another row's; past the window that is looked up.
  const bool row_ends = lane < 31 ? (row_heads >> (lane + 1)) & 1u : p + 1 >= N || __ldcg(ix.keys + p + 1) != my_key;
  if (row_ends) ix.rows[my_key].y = static_cast<uint32_t>(p) + 1u;
}

__global__ void emb_mark_kernel(EmbIndex ix, long long N, int T_len, int V_rows) {
  griddep_enter();
  const long long stride = static_cast<long long>(gridDim.x) * (blockDim.x / 32);
  for (long long w = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32; w * 32 < N; w += stride)
    emb_mark(ix, w * 32, N, static_cast<uint32_t>(T_len), static_cast<uint32_t>(V_rows), lane_id());
}

struct EmbSort {
  const void* ids;
  int index64;
  long long N;
  int V;
  long long padding;
  int passes;            // of BITS bits
  uint32_t* keys[2];     // ping-pong: pass p writes [p & 1]
  uint32_t* toks[2];
  EmbIndex ix;           // its counters and rows are cleared here; CTAS = 1 fills the rest
  int turns;             // counters in ix.turns
  int T;
  uint32_t* status;
};

// Sorts the N tokens by key in stable passes of BITS bits: 8, or 9 where that is a pass less (V of 256 ..
// 511, 2^16 .. 2^18 - 1, from 2^24).  One cluster: every warp owns a contiguous
// range of positions, in (block, warp) order, so the position of its next token of a digit is
// (digits below) + (blocks before) + (warps before) + (its own so far), and blocks exchange only
// their digit totals, through distributed shared memory.  All of this is latency, which one
// launch keeps smallest: with the keys of a pass held in registers, 8 blocks take about 5 us a pass
// at 16384 tokens.  CTAS = 1 serves calls of up to a thousand tokens, where a cluster's barriers would
// cost more than its blocks save.
template <int BITS>
constexpr size_t kEmbSortSmem = sizeof(uint32_t) * (kEmbSortWarps << BITS);
template <int CTAS, int BITS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kEmbSortThreads, 1)
    emb_sort_kernel(const __grid_constant__ EmbSort p) {
  griddep_enter();
  constexpr int kRadix = 1 << BITS;
  constexpr int kParts = kEmbSortThreads / kRadix, kPartWarps = kEmbSortWarps / kParts;
  extern __shared__ uint32_t hist_raw[];
  auto const hist = reinterpret_cast<uint32_t(*)[kRadix]>(hist_raw);  // [warp]: counts, then its next position per digit
  __shared__ uint32_t part_total[kParts][kRadix];  // of kPartWarps warps each
  __shared__ uint32_t total[kRadix];               // this block's digit totals, read by the cluster
  __shared__ uint32_t base[kRadix];
  const int tid = threadIdx.x, warp = tid / 32;
  const uint32_t lane = lane_id();
  const uint32_t rank = CTAS > 1 ? cluster_rank() : 0u;
  const int digit = tid % kRadix, part = tid / kRadix;
  const uint32_t below = (1u << lane) - 1u;
  auto sync_all = [] {
    if constexpr (CTAS > 1) {
      __syncwarp();
      cluster_sync_all();
    } else {
      __syncthreads();
    }
  };

  const long long per = ((p.N + CTAS * kEmbSortWarps - 1) / (CTAS * kEmbSortWarps) + 31) / 32 * 32;
  const long long w0 = (static_cast<long long>(rank) * kEmbSortWarps + warp) * per;
  const long long begin = w0 < p.N ? w0 : p.N;
  const long long end = begin + per < p.N ? begin + per : p.N;
  constexpr int kHeld = 4;  // keys a thread keeps through a pass (N up to CTAS * 4096)
  const bool held = per <= 32 * kHeld;

  if (rank == 0 && tid == 0) {
    *p.status = 0u;
    *p.ix.heavies = 0u;
    *p.ix.longs = 0u;
  }
  for (long long v = static_cast<long long>(rank) * kEmbSortThreads + tid; v < p.V; v += CTAS * kEmbSortThreads)
    p.ix.rows[v] = make_uint2(0u, 0u);
  for (int c = static_cast<int>(rank) * kEmbSortThreads + tid; c < p.turns; c += CTAS * kEmbSortThreads) p.ix.turns[c] = 0u;
  sync_all();  // the status word is cleared before a key may set it

  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = BITS * pass;
    const uint32_t* kin = (pass & 1) ? p.keys[0] : p.keys[1];
    const uint32_t* tin = (pass & 1) ? p.toks[0] : p.toks[1];
    uint32_t* kout = (pass & 1) ? p.keys[1] : p.keys[0];
    uint32_t* tout = (pass & 1) ? p.toks[1] : p.toks[0];
    auto key_at = [&](long long at) {
      return pass ? __ldcg(kin + at) : emb_key(p.ids, p.index64, at, p.V, p.padding, p.status);
    };
    auto tok_at = [&](long long at) { return pass ? __ldcg(tin + at) : static_cast<uint32_t>(at); };
    uint32_t hk[kHeld], ht[kHeld];
    if (held) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const long long at = begin + 32 * i + lane;
        hk[i] = at < end ? key_at(at) : 0u;
        ht[i] = at < end ? tok_at(at) : 0u;
      }
    }
    for (int q = tid; q < kEmbSortWarps * kRadix; q += kEmbSortThreads) hist_raw[q] = 0u;
    __syncthreads();
    if (held) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (begin + 32 * i + lane < end) atomicAdd(&hist[warp][(hk[i] >> shift) & (kRadix - 1)], 1u);
    } else {
      for (long long at = begin + lane; at < end; at += 32)
        atomicAdd(&hist[warp][(key_at(at) >> shift) & (kRadix - 1)], 1u);
    }
    __syncthreads();
    {  // warps before this one, among those of its part
      uint32_t sum = 0;
#pragma unroll
      for (int w = 0; w < kPartWarps; ++w) {
        const uint32_t c = hist[kPartWarps * part + w][digit];
        hist[kPartWarps * part + w][digit] = sum;
        sum += c;
      }
      part_total[part][digit] = sum;
    }
    __syncthreads();
    if (part == 0) {
      uint32_t sum = 0;
#pragma unroll
      for (int q = 0; q < kParts; ++q) sum += part_total[q][digit];
      total[digit] = sum;
    }
    sync_all();
    uint32_t before = 0;
    if (part == 0) {
      uint32_t all = 0;
      if constexpr (CTAS > 1) {
#pragma unroll
        for (uint32_t r = 0; r < CTAS; ++r) {
          const uint32_t c = ld_cluster_u32(smem_addr(&total[digit]), r);
          all += c;
          if (r < rank) before += c;
        }
      } else {
        all = total[digit];
      }
      base[digit] = all;
    }
    __syncthreads();
    if (warp == 0) {  // exclusive sum of the digit totals, kPer digits a lane
      constexpr int kPer = kRadix / 32;
      uint32_t c[kPer], sum = 0;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        c[e] = sum;
        sum += base[kPer * lane + e];
      }
      uint32_t run = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, run, o);
        if (lane >= static_cast<uint32_t>(o)) run += x;
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) base[kPer * lane + e] = run - sum + c[e];
    }
    __syncthreads();
    if (part == 0) base[digit] += before;
    __syncthreads();
    {
      uint32_t b = base[digit];
      for (int q = 0; q < part; ++q) b += part_total[q][digit];
#pragma unroll
      for (int w = 0; w < kPartWarps; ++w) hist[kPartWarps * part + w][digit] += b;
    }
    __syncthreads();
    auto place = [&](bool ok, uint32_t key, uint32_t tok) {
      const uint32_t dg = ok ? (key >> shift) & (kRadix - 1) : kRadix;  // a lane without a token: no digit
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, dg);
      uint32_t pos = 0;
      if (ok) pos = hist[warp][dg] + __popc(same & below);
      __syncwarp();
      if (ok && (same & below) == 0u) hist[warp][dg] += __popc(same);
      __syncwarp();
      if (ok && DP_DCHECK(static_cast<long long>(pos) < p.N, 41u, p.status)) {
        __stcg(kout + pos, key);
        __stcg(tout + pos, tok);
      }
    };
    if (held) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (begin + 32 * i < end) place(begin + 32 * i + lane < end, hk[i], ht[i]);
    } else {
      for (long long at0 = begin; at0 < end; at0 += 32) {
        const bool ok = at0 + lane < end;
        place(ok, ok ? key_at(at0 + lane) : 0u, ok ? tok_at(at0 + lane) : 0u);
      }
    }
    sync_all();  // the pass's arrays are whole, and `total` is free
  }
  if constexpr (CTAS == 1) {
    for (long long w0 = 32 * warp; w0 < p.N; w0 += 32 * kEmbSortWarps)
      emb_mark(p.ix, w0, p.N, static_cast<uint32_t>(p.T), static_cast<uint32_t>(p.V), lane);
  }
}

// ------------------------------------------------------------------------------------- norms
// A chunk of a row in this kernel: kEmbVecs vectors of 16 bytes a lane, four rows of them in flight.  The
// kernel is a stream of dY rows and a warp needs bytes in flight: one sorted position a warp, one vector
// a lane and a barrier between positions took 162 us for 8 x 2048 tokens of 4096 in bf16; this stream takes
// 37 (134 MB at 3.6 TB/s), with two rows in flight 39, with four vectors a lane (half the blocks fit) 42.
// Four blocks an SM leave 64 registers, and the bf16 form spills a little (68 bytes stored, 72 loaded a thread).
constexpr int kEmbVecs = 2;
// Sorted positions whose groups a warp takes.  Fewer spread short calls over more warps (4 x 16 tokens of 64:
// 9.5 us with 16, 7.2 with 4; 16496 of 1032: 18.6 and 16.9; 16384 of 4096: 40 both; with 8: 7.5, 16.3 and 42).
constexpr int kEmbWindow = 4;

// blockIdx.y: chunk.  Long groups first, each by a block whose warps share its rows (all there is to do
// when the norms are given: `short_groups` false).  Then each warp
// takes the short groups that start among kEmbWindow positions: these end within 32, so one load of the
// order shows them all, and their rows are added as one stream, cut where a group ends.
template <typename T>
__global__ void __launch_bounds__(kEmbThreads, 4)
    emb_norm_kernel(const T* __restrict__ dY, long long N, int V_rows, int d, bool short_groups, EmbIndex ix) {
  griddep_enter();
  constexpr int V = EmbVec<T>::N;
  constexpr int kCols = 32 * V * kEmbVecs;
  __shared__ float part[kEmbWarps][kCols];
  const int warp = threadIdx.x / 32;
  const uint32_t lane = lane_id();
  const int chunk = blockIdx.y, chunks = ix.chunks;
  const int col0 = chunk * kCols + static_cast<int>(lane) * V;  // vector v of this lane: col0 + v 32 V
  float acc[kEmbVecs][V];
  auto clear = [&] {
#pragma unroll
    for (int v = 0; v < kEmbVecs; ++v)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[v][e] = 0.0f;
  };
  auto load = [&](uint4 (&q)[kEmbVecs], uint32_t tok, bool ok) {
    const T* row = dY + static_cast<long long>(tok) * d + col0;
#pragma unroll
    for (int v = 0; v < kEmbVecs; ++v) {
      q[v] = make_uint4(0u, 0u, 0u, 0u);
      if (ok && col0 + v * 32 * V < d) q[v] = __ldg(reinterpret_cast<const uint4*>(row + v * 32 * V));
    }
  };
  auto add = [&](const uint4 (&q)[kEmbVecs]) {
#pragma unroll
    for (int v = 0; v < kEmbVecs; ++v) {
      float f[V];
      unpack16(q[v], f, dY);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[v][e] += f[e];
    }
  };
  auto squares = [&] {
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < kEmbVecs; ++v)
#pragma unroll
      for (int e = 0; e < V; ++e) ss = fmaf(acc[v][e], acc[v][e], ss);
    return warp_sum(ss);
  };

  const uint32_t longs = *ix.longs;
  for (uint32_t g = blockIdx.x; g < longs; g += gridDim.x) {
    const uint2 span = ix.long_list[g];
    clear();
    for (uint32_t base = span.x + warp; base < span.y; base += 32 * kEmbWarps) {
      const uint32_t at = base + kEmbWarps * lane;
      const uint32_t tok = at < span.y ? ix.toks[at] : 0u;
      const int rows = static_cast<int>(min((span.y - base + kEmbWarps - 1) / kEmbWarps, 32u));
      for (int k = 0; k < rows; k += 4) {
        uint4 q[4][kEmbVecs];
#pragma unroll
        for (int u = 0; u < 4; ++u) load(q[u], __shfl_sync(0xFFFFFFFFu, tok, (k + u) & 31), k + u < rows);  // 0: absent
#pragma unroll
        for (int u = 0; u < 4; ++u) add(q[u]);
      }
    }
#pragma unroll
    for (int v = 0; v < kEmbVecs; ++v)
#pragma unroll
      for (int e = 0; e < V; ++e) part[warp][(v * V + e) * 32 + lane] = acc[v][e];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int v = 0; v < kEmbVecs; ++v)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float s = 0.0f;
#pragma unroll
          for (int w = 0; w < kEmbWarps; ++w) s += part[w][(v * V + e) * 32 + lane];
          acc[v][e] = s;
        }
      float* out = ix.long_sums + emb_slot(span.x) * d + col0;
#pragma unroll
      for (int v = 0; v < kEmbVecs; ++v) {
        if (col0 + v * 32 * V >= d) continue;
#pragma unroll
        for (int e = 0; e < V / 4; ++e)
          reinterpret_cast<float4*>(out + v * 32 * V)[e] =
              make_float4(acc[v][4 * e], acc[v][4 * e + 1], acc[v][4 * e + 2], acc[v][4 * e + 3]);
      }
      const float ss = squares();
      if (lane == 0) ix.sq[static_cast<long long>(ix.toks[span.x]) * chunks + chunk] = ss;
    }
    __syncthreads();
  }

  if (!short_groups) return;
  const uint32_t none = static_cast<uint32_t>(V_rows);
  const long long windows = (N + kEmbWindow - 1) / kEmbWindow;
  for (long long w = static_cast<long long>(blockIdx.x) * kEmbWarps + warp; w < windows;
       w += static_cast<long long>(gridDim.x) * kEmbWarps) {
    const long long p = w * kEmbWindow + lane;
    const bool in = p < N;
    const int use = in ? ix.use[p] : kEmbHead;
    const uint32_t tok = in ? ix.toks[p] : 0u;
    const bool row = in && (use & kEmbUseMask) == kEmbRow && ix.keys[p] != none;
    const uint32_t heads = __ballot_sync(0xFFFFFFFFu, (use & kEmbHead) != 0);
    const uint32_t rows = __ballot_sync(0xFFFFFFFFu, row);
    if (!(heads & ((1u << kEmbWindow) - 1u))) continue;
    const int a = __ffs(heads) - 1;
    const int z = (heads >> kEmbWindow) ? kEmbWindow + __ffs(heads >> kEmbWindow) - 1 : 32;
    clear();
    uint32_t first = 0;
    for (int k = a; k < z; k += 4) {
      const uint32_t want = (rows >> k) & 15u & (z - k < 4 ? (1u << (z - k)) - 1u : 15u);
      uint4 q[4][kEmbVecs];
      uint32_t t[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) t[u] = __shfl_sync(0xFFFFFFFFu, tok, (k + u) & 31);
      if (!want) continue;
#pragma unroll
      for (int u = 0; u < 4; ++u) load(q[u], t[u], (want >> u) & 1u);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int at = k + u;
        if (!((want >> u) & 1u)) continue;
        if ((heads >> at) & 1u) {
          first = t[u];
          clear();
        }
        add(q[u]);
        if (at + 1 == z || ((heads >> (at + 1)) & 1u)) {
          const float ss = squares();
          if (lane == 0) ix.sq[static_cast<long long>(first) * chunks + chunk] = ss;
        }
      }
    }
  }
}

// |scale| sqrt(sum of a sample's slots), in fp64, by one warp in a fixed order.
__device__ __forceinline__ float emb_norm_by_warp(const float* __restrict__ slots, long long count, float scale,
                                                  uint32_t lane) {
  double acc = 0.0;
#pragma unroll 8
  for (long long k = lane; k < count; k += 32) acc += static_cast<double>(slots[k]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
  return static_cast<float>(fabs(static_cast<double>(scale)) * sqrt(acc));
}

// norms[i] = |scale| sqrt(sum of the sample's T * chunks slots): one block a sample, in a fixed order.
// `by_warp`: in the order above, by one warp, which is what the sum kernel does for itself in small
// calls (kEmbSmallReads), so that every entry point gives a shape's norms in the same bits.
constexpr int kEmbNormThreads = 512;
constexpr long long kEmbSmallReads = 4;
constexpr int kEmbSmallSamples = 64;
__global__ void __launch_bounds__(kEmbNormThreads)
    emb_norms_kernel(const float* __restrict__ sq, long long per_sample, float scale, bool by_warp,
                     float* __restrict__ norms, float* __restrict__ norms_out) {
  griddep_enter();
  __shared__ double part[kEmbNormThreads / 32];
  const float* mine = sq + static_cast<long long>(blockIdx.x) * per_sample;
  if (by_warp) {
    if (threadIdx.x >= 32) return;
    const float n = emb_norm_by_warp(mine, per_sample, scale, threadIdx.x);
    if (threadIdx.x == 0) {
      if (norms) norms[blockIdx.x] = n;
      if (norms_out) norms_out[blockIdx.x] = n;
    }
    return;
  }
  double acc = 0.0;
#pragma unroll 8
  for (long long k = threadIdx.x; k < per_sample; k += kEmbNormThreads) acc += static_cast<double>(mine[k]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kEmbNormThreads / 32; ++w) s += part[w];
    const float n = static_cast<float>(fabs(static_cast<double>(scale)) * sqrt(s));
    if (norms) norms[blockIdx.x] = n;
    if (norms_out) norms_out[blockIdx.x] = n;
  }
}

// --------------------------------------------------------------------------------------- sum
// A lane's 16 bytes of a dY row as quads of columns.
template <typename T>
constexpr int kEmbQuads = EmbVec<T>::N / 4;

__device__ __forceinline__ float4 fma4(float c, float4 x, float4 a) {
  return make_float4(fmaf(c, x.x, a.x), fmaf(c, x.y, a.y), fmaf(c, x.z, a.z), fmaf(c, x.w, a.w));
}

// acc += scale c_i (token's row, or long group's sum) over the sorted positions first .. end.
template <typename T>
__device__ __forceinline__ void emb_add_clipped(const T* __restrict__ dY, const EmbIndex& ix, uint32_t first,
                                                uint32_t end, uint32_t T_len, const float* norms, float C,
                                                float scale, int d, int col, uint32_t lane, float4 (&acc)[kEmbQuads<T>]) {
  constexpr int Q = kEmbQuads<T>;
  constexpr int kU = 4;
  for (uint32_t base = first; base < end; base += 32) {
    const uint32_t at = base + lane;
    const bool in = at < end;
    const uint32_t tok = in ? ix.toks[at] : 0u;
    const int use = in ? ix.use[at] & kEmbUseMask : kEmbSkip;
    const float w = in ? scale * clip_factor(norms[tok / T_len], C) : 0.0f;
    const uint32_t rows = __ballot_sync(0xFFFFFFFFu, use == kEmbRow);
    uint32_t longs = __ballot_sync(0xFFFFFFFFu, use == kEmbLongSum);
    const int count = static_cast<int>(end - base < 32u ? end - base : 32u);
    for (int k0 = 0; k0 < count; k0 += kU) {
      if (!((rows >> k0) & ((1u << kU) - 1u))) continue;
      uint4 q[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t t = __shfl_sync(0xFFFFFFFFu, tok, k0 + u);
        q[u] = make_uint4(0u, 0u, 0u, 0u);
        if (((rows >> (k0 + u)) & 1u) && col < d)
          q[u] = __ldg(reinterpret_cast<const uint4*>(dY + static_cast<long long>(t) * d + col));
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const float c = __shfl_sync(0xFFFFFFFFu, w, k0 + u);
        if (!((rows >> (k0 + u)) & 1u)) continue;
        float f[4 * Q];
        unpack16(q[u], f, dY);
#pragma unroll
        for (int e = 0; e < Q; ++e)
          acc[e] = fma4(c, make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]), acc[e]);
      }
    }
    while (longs) {
      const int k = __ffs(longs) - 1;
      longs &= longs - 1u;
      const float c = __shfl_sync(0xFFFFFFFFu, w, k);
      if (col >= d) continue;
      const float4* sum = reinterpret_cast<const float4*>(ix.long_sums + emb_slot(base + k) * d + col);
#pragma unroll
      for (int e = 0; e < Q; ++e) acc[e] = fma4(c, sum[e], acc[e]);
    }
  }
}

// S[v, :] (+)= its tokens' clipped sums + std z, blockIdx.y: chunk of 32 vectors of 16 bytes.  Heavy
// rows first, each by a block whose warps share its positions; then one row per warp, handed out by
// the chunk's counter (a fixed split left 10% of the SMs' time idle behind the blocks with heavy
// rows).  ACCUMULATE: rows that occur are added to, the others left alone.
// NOISE: Box-Muller tables in shared memory; the normals' arithmetic is then what bounds the
// kernel, the stores of S otherwise.  norms null (small calls): every block forms the B norms from
// the slots itself, which is shorter than another launch, and the first writes norms_out.
template <typename T, bool NOISE, bool ACCUMULATE>
__global__ void __launch_bounds__(kEmbThreads, NOISE ? 4 : 3)
    emb_sum_kernel(const T* __restrict__ dY, EmbIndex ix, int B, int T_len, int V_rows, int d,
                   const float* __restrict__ norms_in, float* __restrict__ norms_out, float C, float scale,
                   double noise_std, PhiloxKey key, uint32_t layer_id, StepRef step, float* __restrict__ S) {
  griddep_enter();
  constexpr int Q = kEmbQuads<T>;
  __shared__ float4 part[kEmbWarps][32 * Q];
  __shared__ double2 tab_s[NOISE ? kNoiseSharedEntries : 1];
  __shared__ float norms_s[kEmbSmallSamples];
  if constexpr (NOISE) stage_noise_tables(tab_s);
  if (!norms_in) {
    const long long per = static_cast<long long>(T_len) * ix.chunks;
    for (int i = threadIdx.x / 32; i < B; i += kEmbWarps) {
      const float n = emb_norm_by_warp(ix.sq + i * per, per, scale, lane_id());
      if (lane_id() == 0) {
        norms_s[i] = n;
        if (norms_out && blockIdx.x == 0 && blockIdx.y == 0) norms_out[i] = n;
      }
    }
  }
  __syncthreads();
  const float* const norms = norms_in ? norms_in : norms_s;
  const uint32_t step_lo = NOISE ? step.get() : 0u;
  const int warp = threadIdx.x / 32;
  const uint32_t lane = lane_id();
  const int col = (blockIdx.y * 32 + static_cast<int>(lane)) * 4 * Q;
  auto store = [&](long long v, float4 (&acc)[Q]) {
    const long long at = v * d + col;
    if constexpr (NOISE) {
      // All quads' normals without a branch between them: their chains interleave.
#pragma unroll
      for (int e = 0; e < Q; ++e) {
        double z[4];
        normals4(static_cast<uint32_t>(static_cast<unsigned long long>(at) / 4) + e, layer_id, step_lo, kStreamNoise,
                 key, z, NoiseTablesShared{tab_s}, noise_std);
        acc[e].x = static_cast<float>(static_cast<double>(acc[e].x) + z[0]);
        acc[e].y = static_cast<float>(static_cast<double>(acc[e].y) + z[1]);
        acc[e].z = static_cast<float>(static_cast<double>(acc[e].z) + z[2]);
        acc[e].w = static_cast<float>(static_cast<double>(acc[e].w) + z[3]);
      }
    }
    if (col >= d || !DP_DCHECK(in_buffer(at, 4 * Q, static_cast<long long>(V_rows) * d), 43u, nullptr)) return;
    float4* out = reinterpret_cast<float4*>(S + at);
#pragma unroll
    for (int e = 0; e < Q; ++e) {
      if constexpr (ACCUMULATE) acc[e] = fma4(1.0f, out[e], acc[e]);
      out[e] = acc[e];
    }
  };
  const uint32_t heavy = *ix.heavies;
  for (uint32_t h = blockIdx.x; h < heavy; h += gridDim.x) {
    const uint32_t v = ix.heavy_list[h];
    const uint2 row = ix.rows[v];
    const uint32_t share = (row.y - row.x + kEmbWarps) / kEmbWarps;  // (positions + warps - 1) / warps
    const uint32_t first = row.x - 1u + share * warp;
    float4 acc[Q] = {};
    emb_add_clipped(dY, ix, first, min(first + share, row.y), static_cast<uint32_t>(T_len), norms, C, scale, d, col, lane,
                    acc);
#pragma unroll
    for (int e = 0; e < Q; ++e) part[warp][e * 32 + lane] = acc[e];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int e = 0; e < Q; ++e) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kEmbWarps; ++w) s = fma4(1.0f, part[w][e * 32 + lane], s);
        acc[e] = s;
      }
      store(v, acc);
    }
    __syncthreads();
  }
  // A turn is a few rows, `turns` apart: ids near each other are often alike in frequency (common
  // ones first), and a warp that took 8 neighbours would have all the long rows.
  const long long warps = static_cast<long long>(gridDim.x) * kEmbWarps;
  // Up to 8 rows, and two turns a warp; but at most 8192 turns where that leaves less than 8, since they queue on
  // the counter at about one a nanosecond (512 tokens of 64, V = 32000, a row a turn: 49 us a step, now 33).
  const long long share = V_rows / (2 * warps);
  const int count = share >= 8 ? 8 : max(static_cast<int>(share), (V_rows + 8191) / 8192);  // below 32
  const long long turns = (V_rows + count - 1) / count;
  for (;;) {
    uint32_t turn = lane == 0 ? atomicAdd(ix.turns + blockIdx.y, 1u) : 0u;
    turn = __shfl_sync(0xFFFFFFFFu, turn, 0);
    if (turn >= turns) break;
    const long long mine = turn + lane * turns;
    const uint2 entry = lane < count && mine < V_rows ? ix.rows[mine] : make_uint2(0u, 0u);
    for (int k = 0; k < count; ++k) {
      const long long v = turn + k * turns;
      if (v >= V_rows) break;
      const uint32_t first = __shfl_sync(0xFFFFFFFFu, entry.x, k), end = __shfl_sync(0xFFFFFFFFu, entry.y, k);
      float4 acc[Q] = {};
      if (first) {
        if (end - first >= kEmbHeavyRow) continue;  // end - (first - 1) tokens: more than kEmbHeavyRow
        emb_add_clipped(dY, ix, first - 1u, end, static_cast<uint32_t>(T_len), norms, C, scale, d, col, lane, acc);
      } else if (ACCUMULATE) {
        continue;
      }
      store(v, acc);
    }
  }
}

}  // namespace dpclip
