// Host side of the embedding entry points: checks, workspace layout and launches.  Included by
// dpclip.cu after its launch helpers.
#pragma once

namespace {

struct EmbCall {
  int B, T, V, d;
  dp_dtype dt;
  long long N() const { return static_cast<long long>(B) * T; }
  int vec() const { return dt == DP_BF16 ? 8 : 4; }
  int chunks() const { return ceil_div(d, 32 * vec()); }                       // of the sum kernel
  // Reads that follow one another where a block's 8 warps form all norms, 8 of 32 slots at a time.
  bool small() const {
    const long long each = (static_cast<long long>(T) * norm_chunks() + 255) / 256;
    return B <= kEmbSmallSamples && ceil_div(B, kEmbWarps) * each <= kEmbSmallReads;
  }
  int norm_chunks() const { return ceil_div(d, 32 * vec() * kEmbVecs); }  // of the norm kernel
};

bool valid_index(dp_index it) { return it == DP_I32 || it == DP_I64; }

bool valid_embedding(const EmbCall& s) {
  if (!valid_dtype(s.dt) || s.B < 1 || s.T < 1 || s.V < 1 || s.d < 1 || s.V == INT32_MAX) return false;
  if (s.d % (s.dt == DP_BF16 ? 8 : 4)) return false;
  if (s.N() >= (1ll << 31)) return false;
  if (static_cast<long long>(s.V) * s.d > (1ll << 34)) return false;
  return s.chunks() <= 65535;
}

struct EmbLayout {
  size_t keys[2], toks[2], rows, use, heavy_list, long_list, turns, sq, long_sums, norms, total;
};

// The counts of heavy rows and long groups share the status word's 256 bytes.
constexpr size_t kEmbHeaviesOffset = 128, kEmbLongsOffset = 132;

EmbLayout emb_layout(const EmbCall& s) {
  EmbLayout L{};
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align256(bytes);
    return o;
  };
  const size_t N = static_cast<size_t>(s.N());
  for (int k = 0; k < 2; ++k) {
    L.keys[k] = take(N * 4);
    L.toks[k] = take(N * 4);
  }
  L.rows = take(static_cast<size_t>(s.V) * sizeof(uint2));
  L.use = take(N);
  L.heavy_list = take((N / (kEmbHeavyRow + 1) + 1) * 4);  // a heavy row has at least kEmbHeavyRow + 1 tokens
  L.long_list = take(static_cast<size_t>(emb_slot(s.N()) + 1) * sizeof(uint2));
  L.turns = take(static_cast<size_t>(s.chunks()) * 4);
  L.sq = take(N * s.norm_chunks() * 4);
  L.long_sums = take(static_cast<size_t>(emb_slot(s.N()) + 1) * s.d * 4);
  L.norms = take(static_cast<size_t>(s.B) * 4);
  L.total = at;
  return L;
}

EmbIndex emb_index(const EmbCall& s, const EmbLayout& L, uint8_t* ws, int passes) {
  auto u32 = [&](size_t o) { return reinterpret_cast<uint32_t*>(ws + o); };
  EmbIndex ix{};
  const int last = (passes - 1) & 1;
  ix.keys = u32(L.keys[last]);
  ix.toks = u32(L.toks[last]);
  ix.heavies = u32(kEmbHeaviesOffset);
  ix.heavy_list = u32(L.heavy_list);
  ix.longs = u32(kEmbLongsOffset);
  ix.long_list = reinterpret_cast<uint2*>(ws + L.long_list);
  ix.turns = u32(L.turns);
  ix.chunks = s.norm_chunks();
  ix.rows = reinterpret_cast<uint2*>(ws + L.rows);
  ix.use = ws + L.use;
  ix.sq = reinterpret_cast<float*>(ws + L.sq);
  ix.long_sums = reinterpret_cast<float*>(ws + L.long_sums);
  return ix;
}

// Up to this many tokens one block sorts them and marks the order (512 tokens: 18.7 us a step against 20.1 with
// a cluster and the marks' own launch; 1024: 22.7 and 23.5; 2048: 28.0 and 25.4; 4096: 38 and 29).
constexpr long long kEmbSortAlone = 1024;

// Grid of the norm and sum kernels: x over warps' items, y over chunks, `per_sm` blocks an SM.
dim3 emb_grid(int chunks, long long items, int per_sm) {
  const long long want = static_cast<long long>(sm_count()) * per_sm / chunks;
  const long long most = (items + kEmbWarps - 1) / kEmbWarps;
  const long long x = std::max(1ll, std::min(want, most));
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(chunks));
}

// The stable passes of `bits` bits that order keys 0 .. V, V itself being the key of a token without a group.
int emb_passes(int V, int bits) {
  int passes = 1;
  while ((static_cast<unsigned long long>(V) >> (bits * passes)) != 0) ++passes;
  return passes;
}
int emb_digit_bits(int V) { return emb_passes(V, 9) < emb_passes(V, 8) ? 9 : 8; }

template <int CTAS, int BITS>
dp_status emb_sort_launch(const EmbSort& p, cudaStream_t stream) {
  if constexpr (BITS > 8) {  // past 48 KB with the static arrays
    static std::atomic<bool> configured[64] = {};
    int dev = 0;
    DP_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64 || !configured[dev].load()) {
      DP_CUDA(cudaFuncSetAttribute(emb_sort_kernel<CTAS, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(kEmbSortSmem<BITS>)));
      if (dev >= 0 && dev < 64) configured[dev].store(true);
    }
  }
  LaunchScope scope(kKindEmbSort, stream);
  DP_LAUNCH("emb_sort_kernel", (emb_sort_kernel<CTAS, BITS>), CTAS, kEmbSortThreads, kEmbSortSmem<BITS>, stream, p);
  return DP_OK;
}

dp_status emb_sort(const EmbCall& s, const EmbLayout& L, const EmbIndex& ix, int passes, const void* ids, dp_index it,
                   long long padding, uint8_t* ws, cudaStream_t stream) {
  EmbSort p{};
  p.ids = ids;
  p.index64 = it == DP_I64 ? 1 : 0;
  p.N = s.N();
  p.V = s.V;
  p.padding = padding;
  p.passes = passes;
  for (int k = 0; k < 2; ++k) {
    p.keys[k] = reinterpret_cast<uint32_t*>(ws + L.keys[k]);
    p.toks[k] = reinterpret_cast<uint32_t*>(ws + L.toks[k]);
  }
  p.ix = ix;
  p.turns = s.chunks();
  p.T = s.T;
  p.status = reinterpret_cast<uint32_t*>(ws);
  const bool wide = emb_digit_bits(s.V) == 9;
  if (p.N <= kEmbSortAlone) return wide ? emb_sort_launch<1, 9>(p, stream) : emb_sort_launch<1, 8>(p, stream);
  const dp_status st = wide ? emb_sort_launch<8, 9>(p, stream) : emb_sort_launch<8, 8>(p, stream);
  if (st != DP_OK) return st;
  LaunchScope scope(kKindEmbSort, stream);
  DP_LAUNCH("emb_mark_kernel", emb_mark_kernel, stream_grid(static_cast<unsigned long long>(p.N), 128), 128, 0, stream, ix,
            p.N, s.T, s.V);
  return DP_OK;
}

dp_status emb_group_sums(const EmbCall& s, const EmbIndex& ix, const void* dY, bool short_groups, cudaStream_t stream) {
  const dim3 grid = emb_grid(s.norm_chunks(), (s.N() + kEmbWindow - 1) / kEmbWindow, 8);
  LaunchScope scope(kKindEmbNorm, stream);
  if (s.dt == DP_BF16) {
    DP_LAUNCH("emb_norm_kernel", emb_norm_kernel<__nv_bfloat16>, grid, kEmbThreads, 0, stream,
              static_cast<const __nv_bfloat16*>(dY), s.N(), s.V, s.d, short_groups, ix);
  } else {
    DP_LAUNCH("emb_norm_kernel", emb_norm_kernel<float>, grid, kEmbThreads, 0, stream, static_cast<const float*>(dY),
              s.N(), s.V, s.d, short_groups, ix);
  }
  return DP_OK;
}

dp_status emb_norms(const EmbCall& s, const EmbIndex& ix, float scale, float* norms, float* norms_out,
                    cudaStream_t stream) {
  LaunchScope scope(kKindFinalize, stream);
  DP_LAUNCH("emb_norms_kernel", emb_norms_kernel, s.B, kEmbNormThreads, 0, stream, ix.sq,
            static_cast<long long>(s.T) * s.norm_chunks(), scale, s.small(), norms, norms_out);
  return DP_OK;
}

template <typename T>
dp_status emb_sum_as(const EmbCall& s, const EmbIndex& ix, const T* dY, const float* norms, float* norms_out, float C,
                     float scale, bool accumulate, double noise_std, unsigned long long seed, StepRef step, unsigned layer_id,
                     float* S, cudaStream_t stream) {
  const PhiloxKey key = philox_key_from_seed(seed);
  LaunchScope scope(kKindEmbSum, stream);
  if (accumulate) {
    DP_LAUNCH("emb_sum_kernel", (emb_sum_kernel<T, false, true>), emb_grid(s.chunks(), s.V, 8), kEmbThreads, 0, stream,
              dY, ix, s.B, s.T, s.V, s.d, norms, norms_out, C, scale, 0.0, key, layer_id, step, S);
  } else if (noise_std != 0.0) {
    DP_LAUNCH("emb_sum_kernel", (emb_sum_kernel<T, true, false>), emb_grid(s.chunks(), s.V, 4), kEmbThreads, 0, stream,
              dY, ix, s.B, s.T, s.V, s.d, norms, norms_out, C, scale, noise_std, key, layer_id, step, S);
  } else {
    DP_LAUNCH("emb_sum_kernel", (emb_sum_kernel<T, false, false>), emb_grid(s.chunks(), s.V, 8), kEmbThreads, 0, stream,
              dY, ix, s.B, s.T, s.V, s.d, norms, norms_out, C, scale, 0.0, key, layer_id, step, S);
  }
  return DP_OK;
}

// norms null (small calls): formed from the slots by the kernel, which then writes norms_out.
dp_status emb_sum(const EmbCall& s, const EmbIndex& ix, const void* dY, const float* norms, float* norms_out, float C,
                  float scale, bool accumulate, double noise_std, unsigned long long seed, StepRef step, unsigned layer_id, float* S,
                  cudaStream_t stream) {
  if (s.dt == DP_BF16)
    return emb_sum_as(s, ix, static_cast<const __nv_bfloat16*>(dY), norms, norms_out, C, scale, accumulate, noise_std, seed,
                      step, layer_id, S, stream);
  return emb_sum_as(s, ix, static_cast<const float*>(dY), norms, norms_out, C, scale, accumulate, noise_std, seed, step,
                    layer_id, S, stream);
}

// Checks shared by the gradient entry points; fills the layout and the number of sort passes.
dp_status emb_check(const EmbCall& s, const void* ids, dp_index it, const void* dY, float scale, void* workspace,
                    size_t ws_bytes, EmbLayout* L, int* passes) {
  if (!ids || !dY || !workspace || !valid_index(it)) return DP_ERR_INVALID_ARG;
  if (!aligned16(dY) || (reinterpret_cast<uintptr_t>(ids) & (it == DP_I64 ? 7u : 3u)) != 0) return DP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return DP_ERR_INVALID_ARG;
  if (!valid_embedding(s) || !std::isfinite(scale)) return DP_ERR_INVALID_ARG;
  *L = emb_layout(s);
  if (ws_bytes < L->total) return DP_ERR_WORKSPACE;
  *passes = emb_passes(s.V, emb_digit_bits(s.V));
  return DP_OK;
}

// Rows of at least this many elements are looked up a warp at a time.
constexpr int kEmbWideRow = 512;

template <typename TI, typename TO>
dp_status emb_lookup_as(const void* W, const void* ids, dp_index it, float scale, long long N, int V, int d, void* Y,
                        cudaStream_t stream) {
  const int wide = sizeof(TI) == 4 && sizeof(TO) == 4 && d % 8 ? 4 : 8;
  // Four vectors a thread: enough blocks that every SM holds 2048 threads, and no more.
  const long long vecs = N * (d / wide);
  const int grid = stream_grid(static_cast<unsigned long long>((vecs + 3) / 4), 256);
  LaunchScope scope(kKindEmbLookup, stream);
  if (wide == 8 && d >= kEmbWideRow && d <= 65535 * 1024) {
    const int segments = ceil_div(d, 1024);
    const long long rows = std::max(1ll, std::min((N + 7) / 8, static_cast<long long>(sm_count()) * 32 / segments));
    DP_LAUNCH("emb_lookup_wide_kernel", (emb_lookup_wide_kernel<TI, TO>),
              dim3(static_cast<unsigned>(rows), static_cast<unsigned>(segments)), 256, 0, stream, static_cast<const TI*>(W),
              ids, it == DP_I64 ? 1 : 0, scale, N, V, d, static_cast<TO*>(Y));
    return DP_OK;
  }
  if constexpr (sizeof(TI) == 4 && sizeof(TO) == 4) {
    if (wide == 4) {
      DP_LAUNCH("emb_lookup_kernel", (emb_lookup_kernel<TI, TO, 4>), grid, 256, 0, stream, static_cast<const TI*>(W), ids,
                it == DP_I64 ? 1 : 0, scale, N, V, d, static_cast<TO*>(Y));
      return DP_OK;
    }
  }
  DP_LAUNCH("emb_lookup_kernel", (emb_lookup_kernel<TI, TO, 8>), grid, 256, 0, stream, static_cast<const TI*>(W), ids,
            it == DP_I64 ? 1 : 0, scale, N, V, d, static_cast<TO*>(Y));
  return DP_OK;
}

dp_status embedding_step(const void* ids, dp_index it, const void* dY, dp_dtype dt, int B, int T, int V, int d,
                         float scale, long long padding_idx, float C, float sigma, unsigned long long seed, StepRef step,
                         unsigned layer_id, float* norms_out, float* G_out, void* workspace, size_t ws_bytes,
                         void* stream) {
  const EmbCall s{B, T, V, d, dt};
  EmbLayout L;
  int passes;
  dp_status st = emb_check(s, ids, it, dY, scale, workspace, ws_bytes, &L, &passes);
  if (st != DP_OK) return st;
  if (!G_out || !aligned16(G_out)) return DP_ERR_INVALID_ARG;
  if (!(C > 0.0f) || !(sigma >= 0.0f) || std::isinf(sigma)) return DP_ERR_INVALID_ARG;
  if (std::isinf(C) && sigma != 0.0f) return DP_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const EmbIndex ix = emb_index(s, L, ws, passes);
  float* norms = reinterpret_cast<float*>(ws + L.norms);
  const double noise_std = (sigma == 0.0f) ? 0.0 : static_cast<double>(sigma) * static_cast<double>(C);
  if ((st = emb_sort(s, L, ix, passes, ids, it, padding_idx, ws, cs)) != DP_OK) return st;
  if ((st = emb_group_sums(s, ix, dY, true, cs)) != DP_OK) return st;
  if (s.small())
    return emb_sum(s, ix, dY, nullptr, norms_out, C, scale, false, noise_std, seed, step, layer_id, G_out, cs);
  if ((st = emb_norms(s, ix, scale, norms, norms_out, cs)) != DP_OK) return st;
  return emb_sum(s, ix, dY, norms, nullptr, C, scale, false, noise_std, seed, step, layer_id, G_out, cs);
}

}  // namespace

extern "C" {

size_t dp_embedding_workspace_size(int B, int T, int V, int d, dp_dtype dt) {
  const EmbCall s{B, T, V, d, dt};
  return valid_embedding(s) ? emb_layout(s).total : 0;
}

dp_status dp_embedding_lookup(const void* W, dp_dtype w_dt, const void* ids, dp_index it, float scale, long long N,
                              int V, int d, void* Y, dp_dtype y_dt, void* stream) {
  DP_NVTX_RANGE();
  if (!W || !ids || !Y || !valid_dtype(w_dt) || !valid_dtype(y_dt) || !valid_index(it)) return DP_ERR_INVALID_ARG;
  if (!aligned16(W) || !aligned16(Y) || (reinterpret_cast<uintptr_t>(ids) & (it == DP_I64 ? 7u : 3u)) != 0)
    return DP_ERR_INVALID_ARG;
  const int q = (w_dt == DP_BF16 || y_dt == DP_BF16) ? 8 : 4;
  if (N < 1 || N >= (1ll << 31) || V < 1 || d < 1 || d % q || !std::isfinite(scale)) return DP_ERR_INVALID_ARG;
  if (static_cast<long long>(V) * d > (1ll << 34)) return DP_ERR_INVALID_ARG;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (w_dt == DP_BF16)
    return y_dt == DP_BF16 ? emb_lookup_as<__nv_bfloat16, __nv_bfloat16>(W, ids, it, scale, N, V, d, Y, cs)
                           : emb_lookup_as<__nv_bfloat16, float>(W, ids, it, scale, N, V, d, Y, cs);
  return y_dt == DP_BF16 ? emb_lookup_as<float, __nv_bfloat16>(W, ids, it, scale, N, V, d, Y, cs)
                         : emb_lookup_as<float, float>(W, ids, it, scale, N, V, d, Y, cs);
}

dp_status dp_embedding_per_sample_norms(const void* ids, dp_index it, const void* dY, dp_dtype dt, int B, int T, int V,
                                        int d, float scale, long long padding_idx, float* norms, void* workspace,
                                        size_t ws_bytes, void* stream) {
  DP_NVTX_RANGE();
  const EmbCall s{B, T, V, d, dt};
  EmbLayout L;
  int passes;
  dp_status st = emb_check(s, ids, it, dY, scale, workspace, ws_bytes, &L, &passes);
  if (st != DP_OK) return st;
  if (!norms) return DP_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const EmbIndex ix = emb_index(s, L, ws, passes);
  if ((st = emb_sort(s, L, ix, passes, ids, it, padding_idx, ws, cs)) != DP_OK) return st;
  if ((st = emb_group_sums(s, ix, dY, true, cs)) != DP_OK) return st;
  return emb_norms(s, ix, scale, nullptr, norms, cs);
}

dp_status dp_embedding_clip_accumulate(const void* ids, dp_index it, const void* dY, dp_dtype dt, int B, int T, int V,
                                       int d, float scale, long long padding_idx, const float* norms, float C,
                                       float* G_sum, void* workspace, size_t ws_bytes, void* stream) {
  DP_NVTX_RANGE();
  const EmbCall s{B, T, V, d, dt};
  EmbLayout L;
  int passes;
  dp_status st = emb_check(s, ids, it, dY, scale, workspace, ws_bytes, &L, &passes);
  if (st != DP_OK) return st;
  if (!norms || !G_sum || !aligned16(G_sum) || !(C > 0.0f)) return DP_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const EmbIndex ix = emb_index(s, L, ws, passes);
  if ((st = emb_sort(s, L, ix, passes, ids, it, padding_idx, ws, cs)) != DP_OK) return st;
  // The long groups' sums are the norm kernel's; the norms themselves are the caller's.
  if ((st = emb_group_sums(s, ix, dY, false, cs)) != DP_OK) return st;
  return emb_sum(s, ix, dY, norms, nullptr, C, scale, true, 0.0, 0, step_value(0), 0, G_sum, cs);
}

dp_status dp_embedding_step(const void* ids, dp_index it, const void* dY, dp_dtype dt, int B, int T, int V, int d,
                            float scale, long long padding_idx, float C, float sigma, unsigned long long seed,
                            unsigned long long step, unsigned layer_id, float* norms_out, float* G_out, void* workspace,
                            size_t ws_bytes, void* stream) {
  DP_NVTX_RANGE();
  return embedding_step(ids, it, dY, dt, B, T, V, d, scale, padding_idx, C, sigma, seed, step_value(step), layer_id,
                        norms_out, G_out, workspace, ws_bytes, stream);
}

dp_status dp_embedding_step_dev_step(const void* ids, dp_index it, const void* dY, dp_dtype dt, int B, int T, int V,
                                     int d, float scale, long long padding_idx, float C, float sigma,
                                     unsigned long long seed, const unsigned long long* step_dev, unsigned layer_id,
                                     float* norms_out, float* G_out, void* workspace, size_t ws_bytes, void* stream) {
  DP_NVTX_RANGE();
  if (!step_dev || (reinterpret_cast<uintptr_t>(step_dev) & 7u) != 0) return DP_ERR_INVALID_ARG;
  return embedding_step(ids, it, dY, dt, B, T, V, d, scale, padding_idx, C, sigma, seed, StepRef{0u, step_dev}, layer_id,
                        norms_out, G_out, workspace, ws_bytes, stream);
}

}  // extern "C"
