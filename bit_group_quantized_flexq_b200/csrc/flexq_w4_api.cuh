// flexq_w4_api.cuh -- host side of the 4-bit linear layers and of the packed
// table's lookup and gradient: argument checks, launch shapes, launches.
#pragma once

#include "flexq_embed.cuh"
#include "flexq_w4.cuh"
#include "flexq_w4_gemm.cuh"

namespace {

int log2_gs(int gs) { return gs == 32 ? 5 : gs == 64 ? 6 : gs == 128 ? 7 : 8; }

// Shapes of the 4-bit form: any N; K a multiple of the group size.
int check_w4_shape(int N, int K, int gs) {
  if (N <= 0 || K <= 0) return fail(FLEXQ_ERR_INVALID_ARG, "sizes must be N > 0, K > 0 (N=%d K=%d)", N, K);
  if (!valid_gs(gs)) return fail(FLEXQ_ERR_UNSUPPORTED, "group_size %d not in {32,64,128,256}", gs);
  if (K % gs) return fail(FLEXQ_ERR_UNSUPPORTED, "K=%d is not a multiple of group_size %d", K, gs);
  if (N > (1 << 30) || K > (1 << 24)) return fail(FLEXQ_ERR_UNSUPPORTED, "N=%d K=%d too large", N, K);
  return FLEXQ_OK;
}

int check_dtype(int dtype) {
  if (dtype != FLEXQ_DTYPE_FP16 && dtype != FLEXQ_DTYPE_BF16)
    return fail(FLEXQ_ERR_INVALID_ARG, "dtype=%d is not FLEXQ_DTYPE_FP16 or FLEXQ_DTYPE_BF16", dtype);
  return FLEXQ_OK;
}

size_t w4_packed_bytes(int N, int K) {
  return static_cast<size_t>(flexq::w4_row_tiles(N)) * flexq::w4_col_tiles(K) * flexq::kW4TileBytes;
}

// ----------------------------------------------------------- linear layers --
constexpr int kGemvTokens = 16;          // batches of the streaming kernel
// and the shared memory it may ask for: an SM's 227 KB less its static arrays
// (the warps' partial sums and the barriers)
constexpr int gemv_smem_limit(int M) {
  return 227 * 1024 - 256 - flexq::gemv_eights(M) * flexq::kGemvWarps * 512;
}

// Lets a kernel use more than 48 KB of shared memory, once per device.
template <typename Kernel>
cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static_assert(kMaxDevices <= 64, "a bit per device");
  if (done.load(std::memory_order_acquire) >> dev & 1) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

cudaLaunchConfig_t gemv_config(unsigned ctas, int split, size_t smem, cudaLaunchAttribute (&attr)[2],
                               cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(flexq::kGemvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  // the first weights are requested while the previous kernel finishes
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cfg;
}

// Clusters of 1, 2, 4 and 8 CTAs with an SM each that the current device runs at
// once, asked once per device; 0 where it has no place for any (a part of a GPU
// may not).  The streaming kernels all take one CTA per SM.
std::atomic<int> g_cluster_limit{8};     // test hook: larger ones are taken as not available

cudaError_t device_clusters(int sms, int (&clusters)[4]) {
  static int known[kMaxDevices][4];
  static std::atomic<unsigned long long> ready{0};
  const auto kern = flexq::w4_gemv_kernel<__half, 4, 1, false>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = allow_smem(kern, gemv_smem_limit(8), ready);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_dev_mutex);
  if (known[dev][0] == 0) {
    int n[4] = {sms, 0, 0, 0};
    for (int i = 1; i < 4; ++i) {
      cudaLaunchAttribute attr[2];
      cudaLaunchConfig_t cfg = gemv_config(1u << i, 1 << i, gemv_smem_limit(8), attr, nullptr);
      cfg.attrs = attr + 1;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&n[i], kern, &cfg);
      if (e != cudaSuccess) return e;
    }
    memcpy(known[dev], n, sizeof(n));
  }
  const int limit = g_cluster_limit.load();
  for (int i = 0; i < 4; ++i) clusters[i] = 1 << i <= limit ? known[dev][i] : 0;
  return cudaSuccess;
}

// Whether the streaming kernel takes a batch: by its size, and by whether the
// share of its activations of a CTA fits shared memory in some cluster that the
// device has.
bool gemv_takes(int M, int kbs, const int (&clusters)[4]) {
  if (M > kGemvTokens || kbs > (1 << 13)) return false;
  for (int i = 0; i < 4 && 1 << i <= flexq::gemv_chunks(kbs); ++i)
    if (clusters[i] > 0 && flexq::gemv_smem(M, kbs, 1 << i, 1) <= gemv_smem_limit(M)) return true;
  return false;
}

// CTAs of a cluster (1, 2, 4 or 8), clusters of a launch and rounds: the
// fewest chunks for the CTA that has most of them, a round more counted as two
// chunks per warp.
struct GemvPlan {
  int split, clusters, rounds;
  long long smem;
};

bool gemv_plan(const flexq::W4Args& a, int strips, const int (&clusters)[4], GemvPlan* plan) {
  long long best = -1;
  for (int i = 0; i < 4; ++i) {
    const int s = 1 << i, n = std::min(strips, clusters[i]);
    if (n == 0 || s > flexq::gemv_chunks(a.kbs)) continue;
    const long long room = gemv_smem_limit(a.M);
    const int most = (strips + n - 1) / n, share = flexq::gemv_share(a.kbs, s);
    int rounds = 1;
    auto of_a_round = [&] { return (most + rounds - 1) / rounds; };
    while (rounds < most && flexq::gemv_smem(a.M, a.kbs, s, of_a_round()) > room) ++rounds;
    const long long smem = flexq::gemv_smem(a.M, a.kbs, s, of_a_round());
    if (smem > room) continue;
    const long long units = static_cast<long long>(most) * share + (rounds - 1) * 2 * flexq::kGemvWarps;
    if (units > INT32_MAX || (best >= 0 && units >= best)) continue;
    best = units;
    *plan = {s, n, rounds, smem};
  }
  return best > 0;
}

template <typename T, int WPG, int NT>
int launch_gemv(const flexq::W4Layers& L, flexq::W4Args a, const int (&clusters)[4], cudaStream_t stream) {
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = allow_smem(flexq::w4_gemv_kernel<T, WPG, NT, false>, gemv_smem_limit(8 * NT), ready);
  if (e != cudaSuccess) return cuda_fail(e, "4-bit linear set-up");
  GemvPlan p;
  if (!gemv_plan(a, L.strip0[L.n], clusters, &p))
    return fail(FLEXQ_ERR_UNSUPPORTED, "no launch for %d tokens, %d strips, K=%d", a.M, L.strip0[L.n], a.K);
  a.split = p.split;
  a.rounds = p.rounds;
  if (p.rounds > 1) {
    static std::atomic<unsigned long long> many{0};
    e = allow_smem(flexq::w4_gemv_kernel<T, WPG, NT, true>, gemv_smem_limit(8 * NT), many);
    if (e != cudaSuccess) return cuda_fail(e, "4-bit linear set-up");
  }
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = gemv_config(static_cast<unsigned>(p.clusters * p.split), p.split,
                                             static_cast<size_t>(p.smem), attr, stream);
  e = p.rounds == 1 ? cudaLaunchKernelEx(&cfg, flexq::w4_gemv_kernel<T, WPG, NT, false>, L, a)
                    : cudaLaunchKernelEx(&cfg, flexq::w4_gemv_kernel<T, WPG, NT, true>, L, a);
  return e == cudaSuccess ? FLEXQ_OK : cuda_fail(e, "4-bit linear launch");
}

template <typename T, int NT>
int launch_gemv_gs(int gs, const flexq::W4Layers& L, const flexq::W4Args& a, const int (&clusters)[4],
                   cudaStream_t stream) {
  return gs == 32    ? launch_gemv<T, 1, NT>(L, a, clusters, stream)
         : gs == 64  ? launch_gemv<T, 2, NT>(L, a, clusters, stream)
         : gs == 128 ? launch_gemv<T, 4, NT>(L, a, clusters, stream)
                     : launch_gemv<T, 8, NT>(L, a, clusters, stream);
}

// ---- batches beyond those: the tcgen05 kernel ----
// FP16 or BF16 activations [M, K], rows ldx apart; box = 64 columns (128
// bytes, swizzled) x T rows.  Rows past M and columns past K read as zero.
int encode_w4_x_map(CUtensorMap* map, const void* x, int dtype, int M, int K, long long ldx, int T) {
  auto fn = encode_fn();
  if (!fn) return fail(FLEXQ_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(M)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ldx) * 2};
  cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(T)};
  cuuint32_t estr[2] = {1u, 1u};
  const CUresult r = fn(map, dtype == FLEXQ_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        2, const_cast<void*>(x), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FLEXQ_ERR_CUDA, "cuTensorMapEncodeTiled (X) failed (%d)", static_cast<int>(r));
  return FLEXQ_OK;
}

// The packed form as strips of 16 kbs rows of 64 bytes; box = one tile of 128
// columns of some strips, 64-byte swizzle.  Strips past the last read as zero.
int encode_w4_map(CUtensorMap* map, const void* wp, int N, int kbs, int strips) {
  auto fn = encode_fn();
  if (!fn) return fail(FLEXQ_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[3] = {16u, static_cast<cuuint64_t>(kbs) * 16, static_cast<cuuint64_t>(flexq::w4_row_tiles(N))};
  cuuint64_t strides[2] = {64u, static_cast<cuuint64_t>(kbs) * flexq::kW4TileBytes};
  cuuint32_t box[3] = {16u, 16u, static_cast<cuuint32_t>(strips)};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(wp), dims, strides,
                        box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(FLEXQ_ERR_CUDA, "cuTensorMapEncodeTiled (4-bit weights) failed (%d)", static_cast<int>(r));
  return FLEXQ_OK;
}

// CTAs of a cluster that share a tile's columns: as many as still run in one
// wave (a sixteenth of the machine's places is left, as clusters do not fill
// every group of SMs), each with at least four column tiles; `most` is the
// largest cluster that the device has.
int w4_mma_split(long long tiles, int kbs, long long slots, int most) {
  int split = 1;
  while (split < most && tiles * (split + 1) <= slots * 15 / 16 && kbs >= 4 * (split + 1)) ++split;
  return split;
}

template <typename E, int T, int RB>
int launch_w4_mma(flexq::W4MmaArgs& a, const flexq::W4Layers& L, const void* x, long long ldx, int sms,
                  int most, cudaStream_t stream) {
  using Cfg = flexq::W4MmaCfg<T, RB>;
  constexpr int dtype = std::is_same<E, __half>::value ? FLEXQ_DTYPE_FP16 : FLEXQ_DTYPE_BF16;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = allow_smem(flexq::w4_mma_kernel<E, T, RB>, Cfg::kSmem, ready);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  int rc = encode_w4_x_map(&a.x, x, dtype, a.M, a.K, ldx, T);
  for (int l = 0; !rc && l < L.n; ++l) {
    rc = encode_w4_map(&a.w[l], L.wp[l], L.N[l], a.kbs, 8 * RB);
    a.tile0[l + 1] = a.tile0[l] + (L.N[l] + Cfg::kRows - 1) / Cfg::kRows;
  }
  if (rc) return rc;
  a.token_tiles = (a.M + T - 1) / T;
  const long long tiles = static_cast<long long>(a.tile0[L.n]) * a.token_tiles;
  if (tiles * 8 > INT32_MAX) return fail(FLEXQ_ERR_UNSUPPORTED, "M=%d with so many weight rows is too large", a.M);
  a.first_wave = Cfg::kCtasPerSm * sms;
  a.split = w4_mma_split(tiles, a.kbs, a.first_wave, most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.split));
  cfg.blockDim = dim3(Cfg::kThreads);
  cfg.dynamicSmemBytes = Cfg::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, flexq::w4_mma_kernel<E, T, RB>, a);
  return e == cudaSuccess ? FLEXQ_OK : cuda_fail(e, "4-bit linear launch");
}

template <typename E>
int launch_linear_w4(const flexq::W4Layers& L, const flexq::W4Args& a, int gs, int sms, cudaStream_t s) {
  int clusters[4], most = 1;
  const cudaError_t e = device_clusters(sms, clusters);
  if (e != cudaSuccess) return cuda_fail(e, "4-bit linear set-up");
  if (gemv_takes(a.M, a.kbs, clusters)) {
    return flexq::gemv_eights(a.M) == 1 ? launch_gemv_gs<E, 1>(gs, L, a, clusters, s)
                                        : launch_gemv_gs<E, 2>(gs, L, a, clusters, s);
  }
  for (int i = 1; i < 4; ++i)
    if (clusters[i] > 0) most = 1 << i;
  flexq::W4MmaArgs m;
  memset(&m, 0, sizeof(m));
  m.n = L.n;
  for (int l = 0; l < L.n; ++l) {
    m.ws[l] = L.ws[l];
    m.y[l] = L.y[l];
    m.ldy[l] = L.ldy[l];
    m.N[l] = L.N[l];
  }
  m.M = a.M;
  m.K = a.K;
  m.G = a.G;
  m.kbs = a.kbs;
  m.gs_shift = a.gs_shift;
  m.status = a.status;
  m.wait_limit_ns = a.wait_limit_ns;
  m.stall = a.stall;
  // Two row blocks per CTA bring the activations half as often, once there are
  // tiles enough for a good part of the SMs: 28672 x 8192 at 64 tokens 53 us
  // with two and 68 with one, 11008 x 4096 at 256 tokens 30 and 34, but 1000 x
  // 2048 at 128 tokens 14.5 and 10.4.
  const int T = a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 ? 64 : 128;
  long long tiles = 0;
  for (int l = 0; l < L.n; ++l) tiles += (L.N[l] + 255) / 256;
  const bool two = T >= 32 && tiles * ((a.M + T - 1) / T) * 5 >= sms;
  switch (T) {
    case 16: return launch_w4_mma<E, 16, 1>(m, L, a.x, a.ldx, sms, most, s);
    case 32: return two ? launch_w4_mma<E, 32, 2>(m, L, a.x, a.ldx, sms, most, s)
                        : launch_w4_mma<E, 32, 1>(m, L, a.x, a.ldx, sms, most, s);
    case 64: return two ? launch_w4_mma<E, 64, 2>(m, L, a.x, a.ldx, sms, most, s)
                        : launch_w4_mma<E, 64, 1>(m, L, a.x, a.ldx, sms, most, s);
    default: return two ? launch_w4_mma<E, 128, 2>(m, L, a.x, a.ldx, sms, most, s)
                        : launch_w4_mma<E, 128, 1>(m, L, a.x, a.ldx, sms, most, s);
  }
}

int linear_w4_common(int M, int K, int gs, int dtype, const void* X, long long ldx, int n_layers,
                     const flexq_layer4_t* layers, void* stream) {
  if (n_layers < 1 || n_layers > flexq::kW4MaxLayers)
    return fail(FLEXQ_ERR_INVALID_ARG, "n_layers=%d is not in 1..%d", n_layers, flexq::kW4MaxLayers);
  if (!layers) return fail(FLEXQ_ERR_INVALID_ARG, "layers is NULL");
  if (M < 0) return fail(FLEXQ_ERR_INVALID_ARG, "M=%d is negative", M);
  // a tile of 128 tokens may number 127 behind the last one
  if (M > INT32_MAX - 127) return fail(FLEXQ_ERR_UNSUPPORTED, "M=%d too large", M);
  int rc = check_dtype(dtype);
  if (rc) return rc;
  for (int l = 0; l < n_layers; ++l)
    if ((rc = check_w4_shape(layers[l].N, K, gs))) return rc;
  if (M == 0) return ok();
  const void* xp[] = {X};
  const char* xn[] = {"X"};
  if ((rc = check_ptrs(1, xp, xn))) return rc;
  if (ldx < K) return fail(FLEXQ_ERR_INVALID_ARG, "ldx=%lld is below K=%d", ldx, K);
  if (ldx % 8) return fail(FLEXQ_ERR_MISALIGNED, "ldx=%lld is not a multiple of 8 elements", ldx);
  for (int l = 0; l < n_layers; ++l) {
    const void* ptrs[] = {layers[l].Wq_packed, layers[l].W_scales};
    const char* names[] = {"Wq_packed", "W_scales"};
    if ((rc = check_ptrs(2, ptrs, names))) return rc;
    if (!layers[l].Y) return fail(FLEXQ_ERR_INVALID_ARG, "Y is NULL");
    if (reinterpret_cast<uintptr_t>(layers[l].Y) & 1u)
      return fail(FLEXQ_ERR_MISALIGNED, "Y is not 2-byte aligned");
    if (layers[l].ldy < layers[l].N)
      return fail(FLEXQ_ERR_INVALID_ARG, "ldy=%lld is below N=%d", layers[l].ldy, layers[l].N);
  }
  DeviceState* st = nullptr;
  if ((rc = device_state(&st))) return rc;

  flexq::W4Layers L = {};
  long long strips = 0;
  L.n = n_layers;
  for (int l = 0; l < n_layers; ++l) {
    L.wp[l] = static_cast<const uint4*>(layers[l].Wq_packed);
    L.ws[l] = static_cast<const __half*>(layers[l].W_scales);
    L.y[l] = layers[l].Y;
    L.ldy[l] = layers[l].ldy;
    L.N[l] = layers[l].N;
    L.strip0[l] = static_cast<int>(strips);
    strips += flexq::w4_row_tiles(layers[l].N);
  }
  L.strip0[n_layers] = static_cast<int>(strips);
  flexq::W4Args a = {};
  a.x = X;
  a.ldx = ldx;
  a.M = M;
  a.K = K;
  a.G = K / gs;
  a.kbs = flexq::w4_col_tiles(K);
  a.gs_shift = log2_gs(gs);
  a.status = st->status;
  a.wait_limit_ns = g_wait_limit_ns.load();
  a.stall = g_inject_stall.exchange(0);
  // the kernels number the 16 x 128 tiles of a launch in 32 bits
  if (strips * a.kbs > INT32_MAX) return fail(FLEXQ_ERR_UNSUPPORTED, "%lld x %d weights are too many", strips * 16, K);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = dtype == FLEXQ_DTYPE_FP16 ? launch_linear_w4<__half>(L, a, gs, st->sms, s)
                                 : launch_linear_w4<__nv_bfloat16>(L, a, gs, st->sms, s);
  return rc ? rc : ok();
}

// ------------------------------------------------------------------ tables --
int check_table(long long T, int V, int K, int gs, int bits, int dtype, int id_bytes) {
  if (bits != 4 && bits != 6) return fail(FLEXQ_ERR_INVALID_ARG, "weight_bits=%d is not 4 or 6", bits);
  if (T < 0) return fail(FLEXQ_ERR_INVALID_ARG, "T=%lld is negative", T);
  if (T > INT32_MAX) return fail(FLEXQ_ERR_UNSUPPORTED, "T=%lld too large", T);
  if (id_bytes != 4 && id_bytes != 8) return fail(FLEXQ_ERR_INVALID_ARG, "id_bytes=%d is not 4 or 8", id_bytes);
  int rc = check_dtype(dtype);
  if (rc) return rc;
  return bits == 4 ? check_w4_shape(V, K, gs) : check_gemm_shape(0, V, K, gs);
}

flexq::Table make_table(const void* Wq, const void* Ws, int V, int K, int gs) {
  flexq::Table t;
  t.packed = static_cast<const uint8_t*>(Wq);
  t.scales = static_cast<const __half*>(Ws);
  t.V = V;
  t.K = K;
  t.G = K / gs;
  t.kbs = flexq::w4_col_tiles(K);
  t.gs_shift = log2_gs(gs);
  return t;
}

template <typename T>
void launch_embed(int bits, const flexq::Table& tb, const void* ids, int id_bytes, int tokens,
                  float scale, void* out, dim3 grid, cudaStream_t s) {
  if (bits == 4)
    flexq::embed_kernel<T, 4><<<grid, flexq::kLookThreads, 0, s>>>(tb, ids, id_bytes, tokens, scale, static_cast<T*>(out));
  else
    flexq::embed_kernel<T, 6><<<grid, flexq::kLookThreads, 0, s>>>(tb, ids, id_bytes, tokens, scale, static_cast<T*>(out));
}

// Sorted tokens per CTA: about six CTAs for each of a whole GPU's 148 SMs (and
// not the device's own number, so that sums have one order everywhere and the
// workspace's size needs no device) where there are that many tokens, between 16 (below, runs that several tiles share cost more than the
// CTAs bring) and kSumMaxTile.
int sum_tile(long long T, int K) {
  const long long cols = (K + 2 * flexq::kSumCols - 1) / (2 * flexq::kSumCols);
  const long long tile = T * cols / (6 * 148);
  return static_cast<int>(std::max<long long>(16, std::min<long long>(flexq::kSumMaxTile, tile)));
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

size_t present_bytes(int V) { return align256((static_cast<size_t>(V) + 31) / 32 * sizeof(unsigned)); }

size_t backward_workspace(long long T, int V, int K) {
  if (T <= flexq::kFewTokens) return 0;
  const long long tiles = (T + sum_tile(T, K) - 1) / sum_tile(T, K);
  return 2 * align256(static_cast<size_t>(T) * sizeof(uint2)) + present_bytes(V) +
         static_cast<size_t>(tiles) * 2 * K * sizeof(float);
}

// Bytes of the rows' gradient that are zeroed while the tokens are sorted, and
// of a piece of the rest, which is zeroed beside the sums (8192 tokens, 32000 x
// 4096 in BF16: 73 us; with 64 MB and pieces of 256 KB 79, with 8 MB 75).
constexpr size_t kSortFill = 32u << 20;
constexpr size_t kFillPiece = 64u << 10;

template <typename T, typename TO>
void launch_few(int bits, const flexq::Table& tb, const flexq::FewArgs& f, unsigned grid, cudaStream_t s) {
  if (bits == 4) flexq::embed_few_kernel<T, TO, 4><<<grid, flexq::kSumThreads, 0, s>>>(tb, f);
  else flexq::embed_few_kernel<T, TO, 6><<<grid, flexq::kSumThreads, 0, s>>>(tb, f);
}

template <typename T, typename TO, int BITS>
cudaError_t launch_sums(const flexq::Table& tb, flexq::SumArgs a, cudaStream_t s) {
  static std::atomic<unsigned long long> ready{0};
  constexpr int smem = static_cast<int>(sizeof(flexq::SumRing<BITS>));
  const cudaError_t e = allow_smem(flexq::embed_sum_kernel<T, TO, BITS>, smem, ready);
  if (e != cudaSuccess) return e;
  const unsigned tiles = static_cast<unsigned>((a.T + static_cast<long long>(a.tile) - 1) / a.tile);
  const unsigned pieces = static_cast<unsigned>((tb.K + flexq::kSumCols - 1) / flexq::kSumCols);
  // each launch's set-up overlaps the end of the one before
  cudaLaunchConfig_t cfg = {};
  a.sum_ctas = static_cast<int>(tiles * ((pieces + 1) / 2));
  cfg.gridDim = dim3(static_cast<unsigned>(a.sum_ctas + a.fill_ctas));
  cfg.blockDim = dim3(flexq::kSumThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t sum = cudaLaunchKernelEx(&cfg, flexq::embed_sum_kernel<T, TO, BITS>, tb, a);
  if (sum != cudaSuccess) return sum;           // more than kFewTokens make several tiles
  cfg.gridDim = dim3(tiles, pieces);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, flexq::embed_join_kernel<T, TO, BITS>, tb, a);
}

template <typename T, typename TO>
cudaError_t launch_sums_bits(int bits, const flexq::Table& tb, const flexq::SumArgs& a, cudaStream_t s) {
  return bits == 4 ? launch_sums<T, TO, 4>(tb, a, s) : launch_sums<T, TO, 6>(tb, a, s);
}

}  // namespace

// ===================================================================== ABI ==
extern "C" {

size_t flexq_weight4_packed_bytes(int N, int K, int group_size) {
  if (N <= 0 || K <= 0 || !valid_gs(group_size) || K % group_size || N > (1 << 30) || K > (1 << 24)) return 0;
  return w4_packed_bytes(N, K);
}

int flexq_quantize_weight4(int N, int K, int group_size, const void* W_fp16, void* Wq_packed,
                           void* W_scales_fp16, void* stream) {
  int rc = check_w4_shape(N, K, group_size);
  if (rc) return rc;
  const void* ptrs[] = {W_fp16, Wq_packed, W_scales_fp16};
  const char* names[] = {"W_fp16", "Wq_packed", "W_scales"};
  if ((rc = check_ptrs(3, ptrs, names))) return rc;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const __half* w = static_cast<const __half*>(W_fp16);
  __half* scales = static_cast<__half*>(W_scales_fp16);
  const long long groups = static_cast<long long>(N) * (K / group_size);
  const long long words = static_cast<long long>(w4_packed_bytes(N, K) / 4);
  if ((groups + 7) / 8 > INT32_MAX || (words + 255) / 256 > INT32_MAX)
    return fail(FLEXQ_ERR_UNSUPPORTED, "N=%d K=%d too large", N, K);
  flexq::w4_scale_kernel<<<static_cast<unsigned>((groups + 7) / 8), 256, 0, s>>>(w, scales, groups, group_size);
  flexq::w4_pack_kernel<<<static_cast<unsigned>((words + 255) / 256), 256, 0, s>>>(
      w, scales, static_cast<uint32_t*>(Wq_packed), N, K, flexq::w4_col_tiles(K), group_size, words);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "4-bit quantizer launch");
  return ok();
}

int flexq_linear_w4_exact(int M, int K, int group_size) {
  if (M <= 0 || check_w4_shape(1, K, group_size)) return 0;
  int clusters[4] = {1, 1, 1, 1}, n = 0;      // without a device, those of a whole GPU
  DeviceState* st = nullptr;
  if (cudaGetDeviceCount(&n) != cudaSuccess || n == 0) {
    cudaGetLastError();
    for (int i = 0; i < 4; ++i) clusters[i] = 1 << i <= g_cluster_limit.load();
  } else if (device_state(&st) || device_clusters(st->sms, clusters) != cudaSuccess) {
    return 0;
  }
  return gemv_takes(M, flexq::w4_col_tiles(K), clusters) ? 1 : 0;
}

int flexq_debug_limit_clusters(int most) {
  if (most < 0 || most > 8) return fail(FLEXQ_ERR_INVALID_ARG, "most=%d is not in 0..8", most);
  g_cluster_limit.store(most == 0 ? 8 : most);
  return ok();
}

int flexq_linear_w4(int M, int N, int K, int group_size, int dtype, const void* X, long long ldx,
                    const void* Wq_packed, const void* W_scales, void* Y, long long ldy, void* stream) {
  const flexq_layer4_t layer = {N, Wq_packed, W_scales, Y, ldy};
  return linear_w4_common(M, K, group_size, dtype, X, ldx, 1, &layer, stream);
}

int flexq_linear_w4_group(int M, int K, int group_size, int dtype, const void* X, long long ldx,
                          int n_layers, const flexq_layer4_t* layers, void* stream) {
  return linear_w4_common(M, K, group_size, dtype, X, ldx, n_layers, layers, stream);
}

int flexq_embedding(long long T, int V, int K, int group_size, int weight_bits, int dtype,
                    const void* ids, int id_bytes, const void* Wq_packed, const void* W_scales,
                    float scale, void* out, void* stream) {
  int rc = check_table(T, V, K, group_size, weight_bits, dtype, id_bytes);
  if (rc) return rc;
  if (T == 0) return ok();
  const void* ptrs[] = {Wq_packed, W_scales, out};
  const char* names[] = {"Wq_packed", "W_scales", "out"};
  if ((rc = check_ptrs(3, ptrs, names))) return rc;
  if (!ids) return fail(FLEXQ_ERR_INVALID_ARG, "ids is NULL");
  if (reinterpret_cast<uintptr_t>(ids) % static_cast<unsigned>(id_bytes))
    return fail(FLEXQ_ERR_MISALIGNED, "ids is not %d-byte aligned", id_bytes);
  DeviceState* st = nullptr;
  if ((rc = device_state(&st))) return rc;
  const flexq::Table tb = make_table(Wq_packed, W_scales, V, K, group_size);
  // a CTA's columns by tokens; up to 64 CTAs per SM, so that most take one or
  // two turns (16384 tokens x 8192 with 16 of them 67 us, with 64 62)
  const unsigned cols = static_cast<unsigned>((K + flexq::kLookCols - 1) / flexq::kLookCols);
  const int ahead = flexq::look_ahead(weight_bits);
  const long long turns = (T + ahead - 1) / ahead;
  const dim3 grid(cols, static_cast<unsigned>(std::min<long long>(turns, std::max(1LL, 64LL * st->sms / cols))));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == FLEXQ_DTYPE_FP16)
    launch_embed<__half>(weight_bits, tb, ids, id_bytes, static_cast<int>(T), scale, out, grid, s);
  else
    launch_embed<__nv_bfloat16>(weight_bits, tb, ids, id_bytes, static_cast<int>(T), scale, out, grid, s);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "embedding launch");
  return ok();
}

size_t flexq_embedding_backward_workspace_bytes(long long T, int V, int K) {
  if (T <= 0 || T > INT32_MAX || V <= 0 || V > (1 << 30) || K <= 0 || K > (1 << 24)) return 0;
  return backward_workspace(T, V, K);
}

int flexq_embedding_backward(long long T, int V, int K, int group_size, int weight_bits, int dtype,
                             const void* ids, int id_bytes, const void* dY, const void* Wq_packed,
                             float scale, int table_dtype, void* d_table, float* d_scales,
                             void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_table(T, V, K, group_size, weight_bits, dtype, id_bytes);
  if (rc) return rc;
  if (!d_table && !d_scales) return fail(FLEXQ_ERR_INVALID_ARG, "d_table and d_scales are both NULL");
  if (d_table && table_dtype != dtype && table_dtype != FLEXQ_DTYPE_FP32)
    return fail(FLEXQ_ERR_INVALID_ARG, "table_dtype=%d is neither dY's type nor FLEXQ_DTYPE_FP32", table_dtype);
  if (!aligned16(d_table) || !aligned16(d_scales))
    return fail(FLEXQ_ERR_MISALIGNED, "d_table or d_scales is not 16-byte aligned");
  const size_t need = backward_workspace(T, V, K);
  if (T > 0) {
    const void* ptrs[] = {dY, workspace};
    const char* names[] = {"dY", "workspace"};
    if ((rc = check_ptrs(need ? 2 : 1, ptrs, names))) return rc;
    if (!ids) return fail(FLEXQ_ERR_INVALID_ARG, "ids is NULL");
    if (reinterpret_cast<uintptr_t>(ids) % static_cast<unsigned>(id_bytes))
      return fail(FLEXQ_ERR_MISALIGNED, "ids is not %d-byte aligned", id_bytes);
    if (workspace_bytes < need)
      return fail(FLEXQ_ERR_INVALID_ARG, "workspace of %zu bytes, the call needs %zu", workspace_bytes, need);
  }
  if (d_scales) {
    const void* ptrs[] = {Wq_packed};
    const char* names[] = {"Wq_packed"};
    if ((rc = check_ptrs(1, ptrs, names))) return rc;
  }
  DeviceState* st = nullptr;
  if ((rc = device_state(&st))) return rc;

  const flexq::Table tb = make_table(Wq_packed, nullptr, V, K, group_size);
  const bool wide = d_table && table_dtype == FLEXQ_DTYPE_FP32;
  flexq::SumArgs a = {};
  a.dy = dY;
  a.T = static_cast<int>(T);
  a.scale = scale;
  a.table = d_table;
  a.scales = d_scales;
  if (T <= flexq::kFewTokens) {
    const flexq::FewArgs f = {a, ids, id_bytes};
    const unsigned grid = static_cast<unsigned>(std::min(V, 4 * st->sms));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == FLEXQ_DTYPE_FP16) {
      if (wide) launch_few<__half, float>(weight_bits, tb, f, grid, s);
      else launch_few<__half, __half>(weight_bits, tb, f, grid, s);
    } else {
      if (wide) launch_few<__nv_bfloat16, float>(weight_bits, tb, f, grid, s);
      else launch_few<__nv_bfloat16, __nv_bfloat16>(weight_bits, tb, f, grid, s);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ok() : cuda_fail(e, "embedding gradient launch");
  }
  const size_t item_bytes = align256(static_cast<size_t>(T) * sizeof(uint2));
  char* ws = static_cast<char*>(workspace);
  flexq::SortArgs so = {};
  so.ids = ids;
  so.id_bytes = id_bytes;
  so.T = static_cast<int>(T);
  so.V = V;
  for (so.passes = 1; so.passes < 4 && (static_cast<long long>(V) >> (8 * so.passes)); ++so.passes) {}
  so.buf[0] = reinterpret_cast<uint2*>(ws);
  so.buf[1] = reinterpret_cast<uint2*>(ws + item_bytes);
  const size_t table_bytes =
      d_table ? static_cast<size_t>(V) * K * (table_dtype == FLEXQ_DTYPE_FP32 ? 4 : 2) : 0;
  const size_t scale_elems = d_scales ? static_cast<size_t>(V) * (K / group_size) : 0;
  const size_t row_bytes = table_bytes / static_cast<size_t>(V);
  if (d_table) {
    a.fill_row = static_cast<int>(std::min<size_t>(static_cast<size_t>(V), kSortFill / row_bytes));
    if (a.fill_row < V) {
      const size_t rest = table_bytes - static_cast<size_t>(a.fill_row) * row_bytes;
      a.fill_ctas = static_cast<int>(std::min<size_t>(std::max<size_t>(1, rest / kFillPiece), static_cast<size_t>(V - a.fill_row)));
      so.present = reinterpret_cast<unsigned*>(ws + 2 * item_bytes);
      a.present = so.present;
    }
  }
  so.fill[0] = static_cast<uint4*>(d_table);
  so.fill[1] = reinterpret_cast<uint4*>(d_scales);
  so.fill_n[0] = static_cast<long long>(static_cast<size_t>(a.fill_row) * row_bytes / 16);
  so.fill_n[1] = static_cast<long long>(scale_elems / 4);
  so.tail = d_scales + scale_elems / 4 * 4;
  so.tail_n = static_cast<int>(scale_elems % 4);
  so.clusters_size = T > 1024 ? 8 : 1;
  const long long pieces = so.fill_n[0] + so.fill_n[1];
  const long long fillers = std::max<long long>(1, std::min<long long>(2LL * st->sms, (pieces + 4095) / 4096));
  const int C = so.clusters_size;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(C + (fillers + C - 1) / C * C));
  cfg.blockDim = dim3(flexq::kSortThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, flexq::embed_sort_kernel, so);
  if (e != cudaSuccess) return cuda_fail(e, "token sort launch");

  a.sorted = so.buf[(so.passes - 1) & 1];
  a.tile = sum_tile(T, K);
  a.partial = reinterpret_cast<float*>(ws + 2 * item_bytes + present_bytes(V));
  if (dtype == FLEXQ_DTYPE_FP16)
    e = wide ? launch_sums_bits<__half, float>(weight_bits, tb, a, cfg.stream)
             : launch_sums_bits<__half, __half>(weight_bits, tb, a, cfg.stream);
  else
    e = wide ? launch_sums_bits<__nv_bfloat16, float>(weight_bits, tb, a, cfg.stream)
             : launch_sums_bits<__nv_bfloat16, __nv_bfloat16>(weight_bits, tb, a, cfg.stream);
  if (e != cudaSuccess) return cuda_fail(e, "embedding gradient launch");
  return ok();
}

}  // extern "C"
