// Host side of the Muon entry points: checks, workspace layout and launches.  Included by
// dpclip.cu after its launch helpers.
#pragma once

namespace {

constexpr int kMuonMaxSteps = 32;
constexpr int kMuonMaxSide = 65536;  // of the smaller dimension: its Gram matrix is m x m

bool valid_muon(int rows, int cols) {
  if (rows < 8 || cols < 8 || rows % 8 || cols % 8) return false;
  if (static_cast<long long>(rows) * cols > (1ll << 34)) return false;
  if (std::max(rows, cols) > (1 << 30)) return false;  // the kernels' column numbers, up to a tile past the end, are 32 bits
  return std::min(rows, cols) <= kMuonMaxSide;
}

constexpr int kMuonBlocksPerSm = 8;
constexpr int kMuonMaxBlocks = 148 * kMuonBlocksPerSm;

struct MuonLayout {
  size_t partials, trace, hi[2], lo[2], A, B, total;
};

MuonLayout muon_layout(int rows, int cols) {
  const size_t m = static_cast<size_t>(std::min(rows, cols));
  const size_t mn = static_cast<size_t>(rows) * static_cast<size_t>(cols);
  MuonLayout L;
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align256(bytes);
    return o;
  };
  L.partials = take(kMuonMaxBlocks * sizeof(double));
  L.trace = take((m + 31) / 32 * 4);
  for (int k = 0; k < 2; ++k) {
    L.hi[k] = take(mn * 2);
    L.lo[k] = take(mn * 2);
  }
  L.A = take(m * m * 2);
  L.B = take(m * m * 2);
  L.total = at;
  return L;
}

// fp16 matrix [rows, cols] in boxes of 64 columns (128 bytes, swizzled) by box_rows rows.
dp_status map_f16(CUtensorMap* map, const __half* base, int rows, int cols, uint32_t box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(cols) * 2};
  const cuuint32_t box[2] = {64, box_rows}, step[2] = {1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<__half*>(base), dims, stride, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    return DP_ERR_CUDA;
  }
  return DP_OK;
}

template <class Cfg>
constexpr auto ns_entry() {
  if constexpr (Cfg::PAIR)
    return ns_pair_kernel<Cfg>;
  else
    return ns_kernel<Cfg>;
}

template <class Cfg>
dp_status ns_configure() {
  static std::atomic<bool> configured[64] = {};
  int dev = 0;
  DP_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64 || !configured[dev].load()) {
    DP_CUDA(cudaFuncSetAttribute(ns_entry<Cfg>(), cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES));
    if (dev >= 0 && dev < 64) configured[dev].store(true);
  }
  return DP_OK;
}

template <class Cfg>
dp_status ns_launch(NsParams p, cudaStream_t stream, int shares) {
  const int ctas = Cfg::PAIR ? 2 : 1;
  const int grid = Cfg::SPLIT ? p.num_units * shares : std::min(p.num_units, sm_count() / ctas) * ctas;
  p.early = 2 * grid <= sm_count() ? 1 : 0;
  LaunchScope scope(kKindNsProduct, stream);
  DP_LAUNCH_CLUSTER("ns_kernel", Cfg::SPLIT ? shares : 0, ns_entry<Cfg>(), grid, Cfg::THREADS, Cfg::SMEM_BYTES, stream, p);
  return DP_OK;
}

// The form of a product: 256 x 256 tiles on SM pairs or 128 x 128 on SMs, and the SMs that share a tile.
struct NsForm {
  bool pair;
  int shares, tiles_m, tiles_n, units;
};

template <int KIND>
NsForm ns_form(const NsParams& p) {
  auto units = [&](int tile, int* tm, int* tn) {
    *tm = ceil_div(p.m, tile);
    *tn = ceil_div(p.n, tile);
    const long long u = KIND == kNsApply ? static_cast<long long>(*tm) * *tn : static_cast<long long>(*tm) * (*tm + 1) / 2;
    return static_cast<int>(u);
  };
  int tm2, tn2, tm1, tn1;
  const int u2 = units(256, &tm2, &tn2), u1 = units(128, &tm1, &tn1);
  if constexpr (KIND != kNsApply) {
    // Few tiles: their K blocks (0.28 us each) are shared by 4 or 2 SMs a tile, where that saves more
    // than the exchange of the parts costs (about 2 us).  Clusters of 4 leave some SMs of a group unused:
    // 36 of them did not fit at once (1024 x 1024: 193 us against 140 unsplit), 32 do.
    const int shares = u1 * 4 <= 128 && p.k_blocks >= 16 ? 4 : u1 * 2 <= sm_count() && p.k_blocks >= 24 ? 2 : 1;
    if (shares > 1) return NsForm{false, shares, tm1, tn1, u1};
  }
  // A wave of 256 x 256 tiles on SM pairs and a wave of 128 x 128 tiles on SMs take about as long
  // (each CTA streams 32 KB a K block); the small tiles' epilogue is half as long.
  const bool pair = ceil_div(u2, sm_count() / 2) < ceil_div(u1, sm_count());
  return pair ? NsForm{true, 1, tm2, tn2, u2} : NsForm{false, 1, tm1, tn1, u1};
}

// A product in its form: configured (before the call's first launch), or launched.
template <int KIND>
dp_status ns_product(NsParams p, cudaStream_t stream, bool configure) {
  const NsForm f = ns_form<KIND>(p);
  p.tiles_m = f.tiles_m;
  p.tiles_n = f.tiles_n;
  p.num_units = f.units;
  auto run = [&](auto cfg) {
    using Cfg = decltype(cfg);
    return configure ? ns_configure<Cfg>() : ns_launch<Cfg>(p, stream, f.shares);
  };
  if constexpr (KIND != kNsApply) {
    if (f.shares > 1) return run(NsConfig<false, KIND, true>{});
  }
  return f.pair ? run(NsConfig<true, KIND>{}) : run(NsConfig<false, KIND>{});
}

struct MuonOut {
  __nv_bfloat16* U = nullptr;
  float* W = nullptr;
  float keep = 1.0f, rate = 0.0f;
};

template <typename T, bool MUON>
dp_status ns_small_configure(bool* wide) {
  static std::atomic<int> state[64] = {};  // 1: configured, 2: and clusters of 16 fit
  int dev = 0;
  DP_CUDA(cudaGetDevice(&dev));
  int known = dev >= 0 && dev < 64 ? state[dev].load() : 0;
  if (known == 0) {
    auto kernel = ns_small_kernel<T, MUON>;
    DP_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNsSmallSmem));
    known = 1;
    // A cluster of more than 8 CTAs needs the device's consent and enough SMs in one group of them.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kNsSmallCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = kNsSmallCtas;
    cfg.blockDim = kNsSmallThreads;
    cfg.dynamicSmemBytes = kNsSmallSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0)
      known = 2;
    (void)cudaGetLastError();  // a refusal is an answer here, not an error of the call
    if (dev >= 0 && dev < 64) state[dev].store(known);
  }
  *wide = known == 2;
  return DP_OK;
}

// CTAs of the one-launch form, 0 where it does not serve: more than 128 rows (as m x n), or more
// columns than its CTAs hold.  One CTA while its 256 columns suffice, since several exchange their
// parts of A; then two chunks of 64 columns a CTA where there are CTAs enough.
int ns_small_ctas(int m, int n, bool wide) {
  const int chunks = ceil_div(n, 64);
  if (m > kNsSmallRows) return 0;
  if (chunks <= kNsSmallMaxChunks) return 1;
  if (chunks <= 4 * 2) return 4;
  if (chunks <= 8 * kNsSmallMaxChunks) return 8;
  return wide && chunks <= kNsSmallCtas * kNsSmallMaxChunks ? kNsSmallCtas : 0;
}

template <typename T, bool MUON>
dp_status ns_small(const T* R, const float* M, int rows, int cols, float mu, float gs, bool nesterov, int steps,
                   const MuonOut& out, const double* partials, int count, int ctas, uint32_t* status,
                   cudaStream_t stream) {
  NsSmall p{};
  p.R = R;
  p.M = M;
  p.rows = rows;
  p.cols = cols;
  p.m = std::min(rows, cols);
  p.n = std::max(rows, cols);
  p.mu = mu;
  p.gs = gs;
  p.nesterov = nesterov ? 1 : 0;
  p.partials = partials;
  p.count = count;
  p.steps = steps;
  p.chunks = ceil_div(ceil_div(p.n, 64), ctas);
  p.U = out.U;
  p.W = out.W;
  p.keep = out.keep;
  p.rate = out.rate;
  p.status = status;
  LaunchScope scope(kKindNsProduct, stream);
  DP_LAUNCH_CLUSTER("ns_small_kernel", ctas, (ns_small_kernel<T, MUON>), ctas, kNsSmallThreads, kNsSmallSmem, stream, p);
  return DP_OK;
}

template <typename T, bool MUON>
dp_status muon_run(const T* R, float* M, int rows, int cols, float mu, float gs, bool nesterov, int steps,
                   const MuonOut& out, uint8_t* ws, cudaStream_t stream) {
  const MuonLayout L = muon_layout(rows, cols);
  const bool tall = rows > cols;
  const int m = tall ? cols : rows, n = tall ? rows : cols;
  dp_status st;
  uint32_t* status = reinterpret_cast<uint32_t*>(ws);
  double* partials = reinterpret_cast<double*>(ws + L.partials);
  auto plane = [&](size_t o) { return reinterpret_cast<__half*>(ws + o); };
  const long long total = static_cast<long long>(rows) * cols;
  const long long vecs = total / EmbVec<T>::N;
  const int most = std::min(sm_count() * kMuonBlocksPerSm, kMuonMaxBlocks);
  const int blocks = static_cast<int>(std::min<long long>(most, (vecs + 4 * kMuonThreads - 1) / (4 * kMuonThreads)));

  // What can fail on the host comes first: the first launch changes the caller's momentum.
  bool wide = false;
  if (m <= kNsSmallRows && (st = ns_small_configure<T, MUON>(&wide)) != DP_OK) return st;
  const int ctas = ns_small_ctas(m, n, wide);
  CUtensorMap xk[2] = {}, xn[2] = {}, ak = {}, bk = {};
  NsParams base;
  memset(&base, 0, sizeof(base));
  base.trace = reinterpret_cast<float*>(ws + L.trace);
  base.order = m;
  base.status = status;
  auto products = [&](int s, bool configure) {
    const int x = s & 1;
    NsParams g = base;
    g.tmA = g.tmB = xk[x];
    g.m = g.n = m;
    g.k_blocks = ceil_div(n, 64);
    g.out = plane(L.A);
    if ((st = ns_product<kNsGram>(g, stream, configure)) != DP_OK) return st;
    NsParams q = base;
    q.tmA = q.tmB = ak;
    q.m = q.n = m;
    q.k_blocks = ceil_div(m, 64);
    q.A = plane(L.A);
    q.out = plane(L.B);
    if ((st = ns_product<kNsPoly>(q, stream, configure)) != DP_OK) return st;
    NsParams a = base;
    a.tmA = bk;
    a.tmB = xn[x];
    a.m = m;
    a.n = n;
    a.k_blocks = ceil_div(m, 64);
    a.hi = plane(L.hi[x]);
    a.lo = plane(L.lo[x]);
    a.out = plane(L.hi[x ^ 1]);
    a.out_lo = plane(L.lo[x ^ 1]);
    if (s + 1 == steps) {
      a.out_mode = out.U ? (tall ? kNsUT : kNsU) : (tall ? kNsWT : kNsW);
      a.U = out.U;
      a.W = out.W;
      a.keep = out.keep;
      a.rate = out.rate;
    }
    return ns_product<kNsApply>(a, stream, configure);
  };
  if (!ctas) {
    for (int k = 0; k < 2; ++k) {
      if ((st = map_f16(&xk[k], plane(L.hi[k]), m, n, 128)) != DP_OK) return st;
      if ((st = map_f16(&xn[k], plane(L.hi[k]), m, n, 64)) != DP_OK) return st;
    }
    if ((st = map_f16(&ak, plane(L.A), m, m, 128)) != DP_OK) return st;
    if ((st = map_f16(&bk, plane(L.B), m, m, 128)) != DP_OK) return st;
    if ((st = products(0, true)) != DP_OK) return st;  // every step's products have the same forms
  }

  {
    LaunchScope scope(kKindMuonMomentum, stream);
    DP_LAUNCH("muon_momentum_kernel", (muon_momentum_kernel<T, MUON>), blocks, kMuonThreads, 0, stream, R, M, vecs, mu, gs,
              nesterov ? 1 : 0, partials, status);
  }
  if (ctas)
    return ns_small<T, MUON>(R, M, rows, cols, mu, gs, nesterov, steps, out, partials, blocks, ctas, status, stream);
  {
    LaunchScope scope(kKindMuonPrepare, stream);
    if (tall) {
      const long long tiles = static_cast<long long>(ceil_div(rows, 64)) * ceil_div(cols, 64);
      DP_LAUNCH("muon_prepare_kernel", (muon_prepare_kernel<T, MUON, true>), static_cast<int>(std::min<long long>(tiles, most)),
                kMuonThreads, 0, stream, R, M, rows, cols, mu, gs, nesterov ? 1 : 0, partials, blocks, plane(L.hi[0]),
                plane(L.lo[0]));
    } else {
      const long long want = (total / 2 + 4 * kMuonThreads - 1) / (4 * kMuonThreads);
      DP_LAUNCH("muon_prepare_kernel", (muon_prepare_kernel<T, MUON, false>), static_cast<int>(std::min<long long>(want, most)),
                kMuonThreads, 0, stream, R, M, rows, cols, mu, gs, nesterov ? 1 : 0, partials, blocks, plane(L.hi[0]),
                plane(L.lo[0]));
    }
  }
  for (int s = 0; s < steps; ++s)
    if ((st = products(s, false)) != DP_OK) return st;
  return DP_OK;
}

}  // namespace

extern "C" {

size_t dp_muon_workspace_size(int rows, int cols) { return valid_muon(rows, cols) ? muon_layout(rows, cols).total : 0; }

dp_status dp_orthogonalize(const void* G, dp_dtype dt, int rows, int cols, int steps, void* U, void* workspace,
                           size_t ws_bytes, void* stream) {
  DP_NVTX_RANGE();
  if (!G || !U || !workspace || U == G || !aligned16(G) || !aligned16(U) || !valid_dtype(dt)) return DP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || !valid_muon(rows, cols)) return DP_ERR_INVALID_ARG;
  if (steps < 1 || steps > kMuonMaxSteps) return DP_ERR_INVALID_ARG;
  if (ws_bytes < muon_layout(rows, cols).total) return DP_ERR_WORKSPACE;
  dp_status st;
  if ((st = get_encoder()) != DP_OK) return st;
  MuonOut out;
  out.U = static_cast<__nv_bfloat16*>(U);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (dt == DP_BF16)
    return muon_run<__nv_bfloat16, false>(static_cast<const __nv_bfloat16*>(G), nullptr, rows, cols, 0.f, 1.f, false, steps,
                                          out, ws, cs);
  return muon_run<float, false>(static_cast<const float*>(G), nullptr, rows, cols, 0.f, 1.f, false, steps, out, ws, cs);
}

dp_status dp_muon_step(float* W, const float* R, float* M, int d_in, int d_out, float lr, float momentum, int nesterov,
                       float weight_decay, float grad_scale, float update_scale, int steps, void* workspace,
                       size_t ws_bytes, void* stream) {
  DP_NVTX_RANGE();
  if (!W || !R || !M || !workspace || !aligned16(W) || !aligned16(R) || !aligned16(M)) return DP_ERR_INVALID_ARG;
  if (W == M || W == R || M == R) return DP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || !valid_muon(d_in, d_out)) return DP_ERR_INVALID_ARG;
  if (!(lr >= 0.0f) || std::isinf(lr) || !(momentum >= 0.0f && momentum < 1.0f) || !(weight_decay >= 0.0f) ||
      std::isinf(weight_decay) || !std::isfinite(grad_scale) || !std::isfinite(update_scale))
    return DP_ERR_INVALID_ARG;
  if (steps < 1 || steps > kMuonMaxSteps) return DP_ERR_INVALID_ARG;
  if (ws_bytes < muon_layout(d_in, d_out).total) return DP_ERR_WORKSPACE;
  dp_status st;
  if ((st = get_encoder()) != DP_OK) return st;
  MuonOut out;
  out.W = W;
  out.keep = static_cast<float>(1.0 - static_cast<double>(lr) * static_cast<double>(weight_decay));
  out.rate = static_cast<float>(static_cast<double>(lr) * static_cast<double>(update_scale));
  return muon_run<float, true>(R, M, d_in, d_out, momentum, grad_scale, nesterov != 0, steps, out,
                               static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
