// Host side of the RMS norm entry points: checks, workspace layout and launches.  Included by
// dpclip.cu after its launch helpers.
#pragma once

namespace {

struct NormCall {
  int B, T, d;
  dp_dtype dt;
  long long N() const { return static_cast<long long>(B) * T; }
  int vecs() const { return d / (dt == DP_BF16 ? 8 : 4); }
};

// A row is at most 2048 vectors of 16 bytes: 512 threads hold four each.
constexpr int kNormMaxVecs = 2048;

dp_status check_norm_shape(const NormCall& s) {
  if (!valid_dtype(s.dt) || s.B < 1 || s.T < 1 || s.d < 1 || s.d % (s.dt == DP_BF16 ? 8 : 4)) return DP_ERR_INVALID_ARG;
  if (s.N() >= (1ll << 31) || s.B > 65535) return DP_ERR_INVALID_ARG;
  return s.vecs() > kNormMaxVecs ? DP_ERR_UNSUPPORTED : DP_OK;
}

// The backward's blocks: up to 512 threads, one row at a time.
int norm_threads(const NormCall& s) { return std::min(512, ceil_div(s.vecs(), 32) * 32); }

// Blocks that share an SM: 1024 threads (the kernel's registers allow that many with one vector a
// thread, 512 with more), while two slots each of the three tensors' rows fit in shared memory.
constexpr int kNormRingBytes = 216 * 1024;
int norm_blocks_per_sm(const NormCall& s) {
  const int threads = norm_threads(s);
  const int by_threads = s.vecs() > threads ? 1 : std::min(16, 1024 / threads);
  return std::max(1, std::min(by_threads, kNormRingBytes / (2 * 3 * s.vecs() * 16)));
}

// Parts of a sample in the backward: blocks fill 148 SMs, each part a run of rows.
int norm_parts(const NormCall& s) {
  const long long want = std::max(1, 148 * norm_blocks_per_sm(s) / s.B);
  const int per = static_cast<int>((s.T + want - 1) / want);
  return ceil_div(s.T, per);
}

struct NormLayout {
  size_t parts, per_sample, total;
};

NormLayout norm_layout(const NormCall& s) {
  NormLayout L;
  L.parts = 256;
  L.per_sample = L.parts + align256(static_cast<size_t>(s.B) * norm_parts(s) * s.d * 4);
  L.total = L.per_sample + align256(static_cast<size_t>(s.B) * s.d * 4);
  return L;
}

template <typename T, int TPR, int NV>
dp_status rmsnorm_launch(const NormCall& s, long long rows, const void* X, const void* res, const float* gain, float eps,
                         void* H, void* Y, cudaStream_t stream) {
  constexpr int threads = TPR < 128 ? 128 : TPR;
  const long long blocks = (rows + threads / TPR - 1) / (threads / TPR);
  const long long cap = static_cast<long long>(sm_count()) * (2048 / threads) * 4;
  const unsigned grid = static_cast<unsigned>(std::min(blocks, cap));
  LaunchScope scope(kKindRmsNorm, stream);
  if (res) {
    DP_LAUNCH("rmsnorm_kernel", (rmsnorm_kernel<T, TPR, NV, true>), grid, threads, 0, stream, static_cast<const T*>(X),
              static_cast<const T*>(res), gain, rows, s.d, eps, static_cast<T*>(H), static_cast<T*>(Y));
  } else {
    DP_LAUNCH("rmsnorm_kernel", (rmsnorm_kernel<T, TPR, NV, false>), grid, threads, 0, stream, static_cast<const T*>(X),
              static_cast<const T*>(res), gain, rows, s.d, eps, static_cast<T*>(H), static_cast<T*>(Y));
  }
  return DP_OK;
}

template <typename T>
dp_status rmsnorm_as(const NormCall& s, long long rows, const void* X, const void* res, const float* gain, float eps,
                     void* H, void* Y, cudaStream_t stream) {
  const int v = s.vecs();
  if (v <= 32) return rmsnorm_launch<T, 32, 1>(s, rows, X, res, gain, eps, H, Y, stream);
  if (v <= 128) return rmsnorm_launch<T, 32, 4>(s, rows, X, res, gain, eps, H, Y, stream);
  if (v <= 256) return rmsnorm_launch<T, 128, 2>(s, rows, X, res, gain, eps, H, Y, stream);
  if (v <= 512) return rmsnorm_launch<T, 128, 4>(s, rows, X, res, gain, eps, H, Y, stream);
  if (v <= 1024) return rmsnorm_launch<T, 256, 4>(s, rows, X, res, gain, eps, H, Y, stream);
  return rmsnorm_launch<T, 512, 4>(s, rows, X, res, gain, eps, H, Y, stream);
}

template <typename T, int NV, bool RES>
dp_status rmsnorm_backward_launch(const NormCall& s, const void* H, const float* gain, const void* dY, const void* dres,
                                  float eps, void* dX, float* parts, uint32_t* status, cudaStream_t stream) {
  constexpr int tensors = RES ? 3 : 2;
  const int nparts = norm_parts(s);
  const int per = ceil_div(s.T, nparts);
  const int slot = tensors * s.vecs() * 16;
  const int stages = std::max(2, std::min({kNormStagesMax, per, kNormRingBytes / norm_blocks_per_sm(s) / slot}));
  static std::atomic<bool> configured[64] = {};
  int dev = 0;
  DP_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64 || !configured[dev].load()) {
    DP_CUDA(cudaFuncSetAttribute(rmsnorm_backward_kernel<T, NV, RES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kNormRingBytes));
    if (dev >= 0 && dev < 64) configured[dev].store(true);
  }
  const dim3 grid(static_cast<unsigned>(nparts), static_cast<unsigned>(s.B));
  LaunchScope scope(kKindRmsNormBackward, stream);
  DP_LAUNCH("rmsnorm_backward_kernel", (rmsnorm_backward_kernel<T, NV, RES>), grid, norm_threads(s),
            static_cast<size_t>(stages) * slot, stream, static_cast<const T*>(H), gain, static_cast<const T*>(dY),
            static_cast<const T*>(dres), s.T, s.d, eps, per, stages, static_cast<T*>(dX), parts, status);
  return DP_OK;
}

template <typename T>
dp_status rmsnorm_backward_as(const NormCall& s, const void* H, const float* gain, const void* dY, const void* dres,
                              float eps, void* dX, float* parts, uint32_t* status, cudaStream_t stream) {
  auto run = [&](auto launch_res, auto launch) {
    return dres ? launch_res(s, H, gain, dY, dres, eps, dX, parts, status, stream)
                : launch(s, H, gain, dY, dres, eps, dX, parts, status, stream);
  };
  if (s.vecs() <= 512) return run(rmsnorm_backward_launch<T, 1, true>, rmsnorm_backward_launch<T, 1, false>);
  if (s.vecs() <= 1024) return run(rmsnorm_backward_launch<T, 2, true>, rmsnorm_backward_launch<T, 2, false>);
  return run(rmsnorm_backward_launch<T, 4, true>, rmsnorm_backward_launch<T, 4, false>);
}

dp_status check_norm_backward(const NormCall& s, const void* H, const float* gain, const void* dY, const void* dres,
                              float eps, const void* dX, const void* workspace, size_t ws_bytes, NormLayout* L) {
  if (!H || !gain || !dY || !dX || !workspace) return DP_ERR_INVALID_ARG;
  if (!aligned16(H) || !aligned16(gain) || !aligned16(dY) || !aligned16(dX) || (dres && !aligned16(dres)))
    return DP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return DP_ERR_INVALID_ARG;
  if (dX == H || dX == dY || dX == dres) return DP_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || std::isinf(eps)) return DP_ERR_INVALID_ARG;
  const dp_status st = check_norm_shape(s);
  if (st != DP_OK) return st;
  *L = norm_layout(s);
  return ws_bytes < L->total ? DP_ERR_WORKSPACE : DP_OK;
}

// More parts of a sample, or bytes of them, than these are summed by a launch of their own.  It costs 1 us on
// the GPU and 2 on the host; up to 16 parts the finish takes as long without it (4 x 16 rows of 256: 8.2 us
// and 8.0; 16 rows of 4096: 9.2 and 8.9; 2 x 64 of 1024, 64 parts: 18.1 and 9.7).
constexpr int kFinishParts = 16;
constexpr long long kFinishPartsBytes = 512 << 10;

// dh, every sample's gain gradient and its norm; with S, the clipped sum and the noise too.
dp_status norm_backward(const NormCall& s, const NormLayout& L, const void* H, const float* gain, const void* dY,
                        const void* dres, float eps, void* dX, float* per_sample, float* norms, float C, double noise_std,
                        unsigned long long seed, StepRef step, unsigned layer_id, float* S, uint8_t* ws,
                        cudaStream_t stream) {
  float* parts = reinterpret_cast<float*>(ws + L.parts);
  uint32_t* status = reinterpret_cast<uint32_t*>(ws);
  const dp_status st =
      s.dt == DP_BF16 ? rmsnorm_backward_as<__nv_bfloat16>(s, H, gain, dY, dres, eps, dX, parts, status, stream)
                      : rmsnorm_backward_as<float>(s, H, gain, dY, dres, eps, dX, parts, status, stream);
  if (st != DP_OK) return st;
  int nparts = norm_parts(s);
  if (nparts > kFinishParts || (nparts > 1 && static_cast<long long>(s.B) * nparts * s.d * 4 > kFinishPartsBytes)) {
    const dim3 grid(static_cast<unsigned>(ceil_div(s.d, 128)), static_cast<unsigned>(s.B));
    const int warps = nparts <= 8 ? 4 : nparts <= 32 ? 8 : kPartsWarps;  // two to four parts a warp, or more
    LaunchScope scope(kKindRmsNormGain, stream);
    DP_LAUNCH("rmsnorm_parts_kernel", rmsnorm_parts_kernel, grid, 32 * warps, 0, stream, parts, nparts, s.d, per_sample);
    parts = per_sample;
    nparts = 1;
  }
  LaunchScope scope(kKindRmsNormGain, stream);
  DP_LAUNCH("rmsnorm_finish_kernel", rmsnorm_finish_kernel, kFinishCtas, kFinishThreads, 0, stream, parts, nparts, s.B,
            s.d, per_sample, norms, C, noise_std, philox_key_from_seed(seed), layer_id, step, S);
  return DP_OK;
}

dp_status rmsnorm_step(const void* H, const float* gain, const void* dY, const void* dres, dp_dtype dt, int B, int T,
                       int d, float eps, float C, float sigma, unsigned long long seed, StepRef step, unsigned layer_id,
                       void* dX, float* norms_out, float* G_out, void* workspace, size_t ws_bytes, void* stream) {
  const NormCall s{B, T, d, dt};
  NormLayout L;
  dp_status st = check_norm_backward(s, H, gain, dY, dres, eps, dX, workspace, ws_bytes, &L);
  if (st != DP_OK) return st;
  if (!G_out || !aligned16(G_out)) return DP_ERR_INVALID_ARG;
  if (!(C > 0.0f) || !(sigma >= 0.0f) || std::isinf(sigma)) return DP_ERR_INVALID_ARG;
  if (std::isinf(C) && sigma != 0.0f) return DP_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const double noise_std = (sigma == 0.0f) ? 0.0 : static_cast<double>(sigma) * static_cast<double>(C);
  return norm_backward(s, L, H, gain, dY, dres, eps, dX, reinterpret_cast<float*>(ws + L.per_sample), norms_out, C,
                       noise_std, seed, step, layer_id, G_out, ws, cs);
}

}  // namespace

extern "C" {

dp_status dp_rmsnorm(const void* X, const void* residual, const float* gain, dp_dtype dt, long long rows, int d,
                     float eps, void* H, void* Y, void* stream) {
  DP_NVTX_RANGE();
  if (!X || !gain || !Y || (residual && !H)) return DP_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(gain) || !aligned16(Y) || (residual && (!aligned16(residual) || !aligned16(H))))
    return DP_ERR_INVALID_ARG;
  if (Y == X || Y == residual || (residual && (H == X || H == residual || H == Y))) return DP_ERR_INVALID_ARG;
  if (rows < 1 || rows >= (1ll << 31) || !(eps >= 0.0f) || std::isinf(eps)) return DP_ERR_INVALID_ARG;
  const NormCall s{1, 1, d, dt};
  const dp_status st = check_norm_shape(s);
  if (st != DP_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return dt == DP_BF16 ? rmsnorm_as<__nv_bfloat16>(s, rows, X, residual, gain, eps, H, Y, cs)
                       : rmsnorm_as<float>(s, rows, X, residual, gain, eps, H, Y, cs);
}

size_t dp_rmsnorm_workspace_size(int B, int T, int d, dp_dtype dt) {
  const NormCall s{B, T, d, dt};
  return check_norm_shape(s) == DP_OK ? norm_layout(s).total : 0;
}

dp_status dp_rmsnorm_backward(const void* H, const float* gain, const void* dY, const void* residual_grad, dp_dtype dt,
                              int B, int T, int d, float eps, void* dX, float* per_sample, float* norms,
                              void* workspace, size_t ws_bytes, void* stream) {
  DP_NVTX_RANGE();
  const NormCall s{B, T, d, dt};
  NormLayout L;
  dp_status st = check_norm_backward(s, H, gain, dY, residual_grad, eps, dX, workspace, ws_bytes, &L);
  if (st != DP_OK) return st;
  if (!per_sample || !norms || !aligned16(per_sample)) return DP_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return norm_backward(s, L, H, gain, dY, residual_grad, eps, dX, per_sample, norms, INFINITY, 0.0, 0, step_value(0), 0,
                       nullptr, ws, cs);
}

dp_status dp_rmsnorm_clip_accumulate(const float* per_sample, const float* norms, int B, int d, float C, float* G_sum,
                                     void* stream) {
  DP_NVTX_RANGE();
  if (!per_sample || !norms || !G_sum || !aligned16(per_sample) || !aligned16(G_sum)) return DP_ERR_INVALID_ARG;
  if (B < 1 || d < 1 || d % 4 || !(C > 0.0f)) return DP_ERR_INVALID_ARG;
  if (d > kNormMaxVecs * 8) return DP_ERR_UNSUPPORTED;  // wider than any row of the backward
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  LaunchScope scope(kKindRmsNormGain, cs);
  DP_LAUNCH("rmsnorm_sum_kernel", rmsnorm_sum_kernel, ceil_div(d, 128), kGainSumThreads, 0, cs, per_sample, norms, B, d, C,
            G_sum);
  return DP_OK;
}

dp_status dp_rmsnorm_step(const void* H, const float* gain, const void* dY, const void* residual_grad, dp_dtype dt,
                          int B, int T, int d, float eps, float C, float sigma, unsigned long long seed,
                          unsigned long long step, unsigned layer_id, void* dX, float* norms_out, float* G_out,
                          void* workspace, size_t ws_bytes, void* stream) {
  DP_NVTX_RANGE();
  return rmsnorm_step(H, gain, dY, residual_grad, dt, B, T, d, eps, C, sigma, seed, step_value(step), layer_id, dX,
                      norms_out, G_out, workspace, ws_bytes, stream);
}

dp_status dp_rmsnorm_step_dev_step(const void* H, const float* gain, const void* dY, const void* residual_grad,
                                   dp_dtype dt, int B, int T, int d, float eps, float C, float sigma,
                                   unsigned long long seed, const unsigned long long* step_dev, unsigned layer_id,
                                   void* dX, float* norms_out, float* G_out, void* workspace, size_t ws_bytes,
                                   void* stream) {
  DP_NVTX_RANGE();
  if (!step_dev || (reinterpret_cast<uintptr_t>(step_dev) & 7u) != 0) return DP_ERR_INVALID_ARG;
  return rmsnorm_step(H, gain, dY, residual_grad, dt, B, T, d, eps, C, sigma, seed, StepRef{0u, step_dev}, layer_id, dX,
                      norms_out, G_out, workspace, ws_bytes, stream);
}

}  // extern "C"
