// api_int8.cuh — host side of the 8-bit integer projection (int8.cuh, decode_int8.cuh). Part of flashnorm.cu.
#pragma once

namespace {

constexpr int64_t kInt8MaxK = 131072;  // 127^2 K stays inside int32

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// K ranges per 128-row slab of the decode kernel: two CTAs on every SM, no range without a stage.
int int8_ksplit(int64_t n_rows, int64_t d, int sms) {
  const int64_t slabs = (n_rows + fn::kI8Rows - 1) / fn::kI8Rows, num_kb = (d + 127) / 128;
  return static_cast<int>(std::max<int64_t>(1, std::min(2 * sms / slabs, num_kb)));
}

// How the one-launch decode kernel runs a shape; ranks 0: it does not (the codes of a K range leave too little shared
// memory for the ring, at large d with so many slabs that few ranks fit).
struct Int8Cluster {
  int slabs, rows, ranks, max_kb, stages;
};

Int8Cluster int8_cluster_plan(int64_t M, int64_t d, int64_t n_rows, int sms) {
  Int8Cluster c = {};
  if (M > FN_DECODE_MAX_M) return c;
  const int64_t num_kb = (d + 127) / 128;
  // rows of a slab and ranks (a power of two) that fill the most of two CTAs per SM: N = 12288, d = 4096 takes 128 slabs of
  // 96 rows with 2 ranks. Clusters of 3 leave SMs empty and run in two waves (22 us with 3 ranks of 128 rows there, 15 with 2,
  // 20 with 1 or, in two waves, 4).
  int64_t rows = fn::kI8Rows, ranks = 1, slabs = 0, best = -1;
  for (int64_t r = fn::kI8Rows; r >= 32; r -= 32) {
    const int64_t n = (n_rows + r - 1) / r;
    int64_t k = 1;
    while (2 * k <= std::min<int64_t>({2 * sms / n, num_kb, fn::kI8cMaxRanks})) k *= 2;
    const int64_t filled = n * k <= 2 * sms ? n * k : 0;  // more than one wave: only as whole slabs of 128
    if (filled > best) rows = r, ranks = k, slabs = n, best = filled;
  }
  const int64_t max_kb = (num_kb + ranks - 1) / ranks;
  // two CTAs per SM where the grid needs them (1 KB of each CTA's share is the system's)
  const int64_t budget = slabs * ranks <= sms ? 227 * 1024 : 228 * 1024 / 2 - 1024;
  if (max_kb > 256) return c;
  const int64_t rest = budget - fn::int8_cluster_smem_bytes(static_cast<int>(M), static_cast<int>(max_kb), 0, static_cast<int>(rows));
  const int64_t stages = std::min<int64_t>({rest / (rows * 128), max_kb, 16});
  if (stages < std::min<int64_t>(max_kb, 3)) return c;
  c.slabs = static_cast<int>(slabs);
  c.rows = static_cast<int>(rows);
  c.ranks = static_cast<int>(ranks);
  c.max_kb = static_cast<int>(max_kb);
  c.stages = static_cast<int>(stages);
  return c;
}

// The workspace of one call: where its parts start, and its size.
struct Int8Workspace {
  int64_t counters, rho, xq, part, bytes;
  int slabs, ksplit;  // decode
};

Int8Workspace int8_workspace(int64_t M, int64_t d, int64_t n_rows, int sms) {
  Int8Workspace w = {};
  if (int8_cluster_plan(M, d, n_rows, sms).ranks) return w;
  const bool decode = M <= FN_DECODE_MAX_M;
  const int64_t slabs = (n_rows + fn::kI8Rows - 1) / fn::kI8Rows;
  w.ksplit = decode ? int8_ksplit(n_rows, d, sms) : 1;
  w.slabs = static_cast<int>(decode && w.ksplit > 1 ? slabs : 0);
  w.counters = 0;
  w.rho = round_up(4ll * w.slabs, 256);
  w.xq = w.rho + round_up(4 * M, 256);
  w.part = w.xq + round_up(M * d, 256);
  w.bytes = w.part + (w.ksplit > 1 ? slabs * w.ksplit * M * fn::kI8Rows * 4 : 0);
  return w;
}

fn_status check_int8_shape(int64_t M, int64_t d, int64_t N, bool glu) {
  if (M < 0 || M > kMaxDim) return fail(FN_ERR_INVALID_ARG, "M = %lld out of range", (long long)M);
  if (d < 16 || d > kMaxDim || d % 16 != 0) return fail(FN_ERR_INVALID_ARG, "d = %lld must be a positive multiple of 16", (long long)d);
  if (N < 8 || N > kMaxDim / 2 || N % (glu ? 16 : 8) != 0)
    return fail(FN_ERR_INVALID_ARG, "N = %lld must be a positive multiple of %d", (long long)N, glu ? 16 : 8);
  if (d > kInt8MaxK) return fail(FN_ERR_UNSUPPORTED, "d = %lld: int32 sums hold at most d = %lld", (long long)d, (long long)kInt8MaxK);
  return FN_OK;
}

template <bool GLU, bool OUT_F32>
fn_status launch_int8_pair(const CUtensorMap& ta, const CUtensorMap& tb, const fn::PairGemmParams& p,
                           const fn::Int8EpiParams& ep, int sms, int dev, cudaStream_t s) {
  return launch_pair_gemm<fn::PG_I8, fn::PgJob<false, false, fn::Int8Epi<GLU, OUT_F32>>>(ta, tb, p, ep, sms, dev, s, "int8 GEMM");
}

template <bool GLU, bool OUT_F32>
fn_status launch_int8_decode(const CUtensorMap& tw, const CUtensorMap& tx, const fn::DecodeInt8Params& p, int slabs,
                             int dev, cudaStream_t s) {
  auto kern = fn::k_decode_int8<GLU, OUT_F32>;
  constexpr int smem = fn::decode_int8_smem_bytes();
  static bool configured[kMaxDevices] = {false};
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute (int8 decode)");
    configured[dev] = true;
  }
  cudaError_t e = launch_kernel(kern, dim3(static_cast<unsigned>(slabs * p.ksplit)), dim3(fn::kI8DecThreads), smem, s, 1,
                                tw, tx, p);
  if (e != cudaSuccess) return cuda_fail(e, "int8 decode launch");
  return FN_OK;
}

template <bool GLU, bool OUT_F32>
fn_status launch_int8_cluster(const CUtensorMap& tw, const fn::Int8ClusterParams& p, int slabs, int dev, cudaStream_t s) {
  auto kern = fn::k_decode_int8_cluster<GLU, OUT_F32>;
  static bool configured[kMaxDevices] = {false};
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute (int8 cluster decode)");
    configured[dev] = true;
  }
  cudaError_t e = launch_kernel(kern, dim3(static_cast<unsigned>(slabs * p.ranks)), dim3(fn::kI8cThreads),
                                fn::int8_cluster_smem_bytes(p.M, p.max_kb, p.stages, p.rows), s, p.ranks, tw, p);
  if (e != cudaSuccess) return cuda_fail(e, "int8 cluster decode launch");
  return FN_OK;
}

fn_status run_int8(const void* x, const void* Q, const void* scales, void* y, int64_t M, int64_t d, int64_t N, float eps,
                   int norm, int out_dtype, bool glu, void* workspace, int64_t workspace_bytes, cudaStream_t s) {
  fn_status st = check_int8_shape(M, d, N, glu);
  if (st != FN_OK) return st;
  if (norm != 0 && norm != 1) return fail(FN_ERR_INVALID_ARG, "norm must be 0 or 1");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(FN_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (out_dtype != FN_BF16 && out_dtype != FN_F32) return fail(FN_ERR_INVALID_ARG, "out_dtype %d unknown", out_dtype);
  if (workspace_bytes < 0) return fail(FN_ERR_INVALID_ARG, "workspace_bytes < 0");
  if (M == 0) return FN_OK;
  if ((st = check_ptr(x, "x")) != FN_OK) return st;
  if ((st = check_ptr(Q, "Q")) != FN_OK) return st;
  if ((st = check_ptr(scales, "scales")) != FN_OK) return st;
  if ((st = check_ptr(y, "y")) != FN_OK) return st;
  if (M > FN_DECODE_MAX_M && (st = check_ptr(workspace, "workspace")) != FN_OK) return st;
  int dev = 0;
  const int sms = device_sm_count(&dev);
  if (sms <= 1) return fail(FN_ERR_CUDA, "cannot query the current device");
  const int64_t n_rows = glu ? 2 * N : N;
  const Int8Cluster c = int8_cluster_plan(M, d, n_rows, sms);
  if (c.ranks) {
    CUtensorMap tw;
    if ((st = make_u8_map(&tw, Q, d, n_rows, c.rows)) != FN_OK) return st;
    fn::Int8ClusterParams p;
    p.x = static_cast<const uint16_t*>(x);
    p.y = y;
    p.scale = static_cast<const float*>(scales);
    p.M = static_cast<int>(M);
    p.K = static_cast<int>(d);
    p.num_kb = static_cast<int>((d + 127) / 128);
    p.n_rows = static_cast<int>(n_rows);
    p.n_out = static_cast<int>(N);
    p.ranks = c.ranks;
    p.rows = c.rows;
    p.stages = c.stages;
    p.max_kb = c.max_kb;
    p.eps = eps;
    p.norm = norm;
    const bool f32 = out_dtype == FN_F32;
    if (glu) return f32 ? launch_int8_cluster<true, true>(tw, p, c.slabs, dev, s) : launch_int8_cluster<true, false>(tw, p, c.slabs, dev, s);
    return f32 ? launch_int8_cluster<false, true>(tw, p, c.slabs, dev, s) : launch_int8_cluster<false, false>(tw, p, c.slabs, dev, s);
  }
  if ((st = check_ptr(workspace, "workspace")) != FN_OK) return st;
  const Int8Workspace w = int8_workspace(M, d, n_rows, sms);
  if (workspace_bytes < w.bytes)
    return fail(FN_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)w.bytes);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  unsigned* counters = reinterpret_cast<unsigned*>(base + w.counters);
  float* rho = reinterpret_cast<float*>(base + w.rho);
  int8_t* xq = reinterpret_cast<int8_t*>(base + w.xq);

  // row pass: as few threads per row as hold it in registers
  const int lpr = d <= 32 * 32 ? 32 : d <= 128 * 32 ? 128 : 256;
  const dim3 grid(static_cast<unsigned>((M + 256 / lpr - 1) / (256 / lpr)));
  auto rows = lpr == 32 ? fn::k_int8_rows<32> : lpr == 128 ? fn::k_int8_rows<128> : fn::k_int8_rows<256>;
  cudaError_t e = launch_kernel(rows, grid, dim3(256), 0, s, 1, static_cast<const uint16_t*>(x), xq, rho,
                                static_cast<int>(M), static_cast<int>(d), eps, norm, counters, w.slabs);
  if (e != cudaSuccess) return cuda_fail(e, "int8 row pass launch");

  CUtensorMap tx, tw;
  if (M <= FN_DECODE_MAX_M) {
    if ((st = make_u8_map(&tx, xq, d, M, fn::kI8Tok)) != FN_OK) return st;
    if ((st = make_u8_map(&tw, Q, d, n_rows, fn::kI8Rows)) != FN_OK) return st;
    fn::DecodeInt8Params p;
    p.y = y;
    p.rho = rho;
    p.scale = static_cast<const float*>(scales);
    p.part = reinterpret_cast<int*>(base + w.part);
    p.counters = counters;
    p.M = static_cast<int>(M);
    p.num_kb = static_cast<int>((d + 127) / 128);
    p.n_rows = static_cast<int>(n_rows);
    p.n_out = static_cast<int>(N);
    p.ksplit = w.ksplit;
    const int slabs = static_cast<int>((n_rows + fn::kI8Rows - 1) / fn::kI8Rows);
    const bool f32 = out_dtype == FN_F32;
    if (glu) return f32 ? launch_int8_decode<true, true>(tw, tx, p, slabs, dev, s) : launch_int8_decode<true, false>(tw, tx, p, slabs, dev, s);
    return f32 ? launch_int8_decode<false, true>(tw, tx, p, slabs, dev, s) : launch_int8_decode<false, false>(tw, tx, p, slabs, dev, s);
  }
  const int step = glu ? 64 : 32;  // whole epilogue blocks
  fn::PairGemmParams p;
  plan_pair_gemm(&p, M, n_rows, (d + 127) / 128, sms, step);
  p.early = fn::PG_EARLY_B;  // Q does not depend on the row pass
  if ((st = make_u8_map(&tx, xq, d, M, 128)) != FN_OK) return st;
  if ((st = make_u8_map(&tw, Q, d, n_rows, p.bn / 2)) != FN_OK) return st;
  fn::Int8EpiParams ep;
  ep.y = y;
  ep.rho = rho;
  ep.scale = static_cast<const float*>(scales);
  ep.n_out = static_cast<int>(N);
  const bool f32 = out_dtype == FN_F32;
  if (glu) return f32 ? launch_int8_pair<true, true>(tx, tw, p, ep, sms, dev, s) : launch_int8_pair<true, false>(tx, tw, p, ep, sms, dev, s);
  return f32 ? launch_int8_pair<false, true>(tx, tw, p, ep, sms, dev, s) : launch_int8_pair<false, false>(tx, tw, p, ep, sms, dev, s);
}

}  // namespace

extern "C" {

fn_status flashnorm_fold_weights_int8(const void* W, const void* g, void* Q, void* scales, int64_t d, int64_t N, int glu,
                                      void* stream) {
  g_last_error[0] = '\0';
  if (glu != 0 && glu != 1) return fail(FN_ERR_INVALID_ARG, "glu must be 0 or 1");
  fn_status st = check_int8_shape(0, d, N, false);
  if (st != FN_OK) return st;
  if (glu && N % 32 != 0) return fail(FN_ERR_INVALID_ARG, "GLU needs N = 2F with F %% 16 == 0, got N = %lld", (long long)N);
  if ((st = check_ptr(W, "W")) != FN_OK) return st;
  if ((st = check_ptr(g, "g")) != FN_OK) return st;
  if ((st = check_ptr(Q, "Q")) != FN_OK) return st;
  if ((st = check_ptr(scales, "scales")) != FN_OK) return st;
  dim3 grid(static_cast<unsigned>((N + fn::kFoldTile - 1) / fn::kFoldTile),
            static_cast<unsigned>((d + fn::kFoldTile - 1) / fn::kFoldTile));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_kernel(fn::k_int8_scales, dim3(static_cast<unsigned>((N + 31) / 32)), dim3(256), 0, s, 1,
                                static_cast<const uint16_t*>(W), static_cast<const uint16_t*>(g),
                                static_cast<float*>(scales), static_cast<int>(d), static_cast<int>(N), glu);
  if (e == cudaSuccess)
    e = launch_kernel(fn::k_fold_int8, grid, dim3(256), 0, s, 1, static_cast<const uint16_t*>(W),
                      static_cast<const uint16_t*>(g), static_cast<const float*>(scales), static_cast<int8_t*>(Q),
                      static_cast<int>(d), static_cast<int>(N), glu);
  if (e != cudaSuccess) return cuda_fail(e, "int8 fold launch");
  return FN_OK;
}

fn_status flashnorm_int8_workspace_bytes(int64_t M, int64_t d, int64_t N, int glu, int64_t* bytes) {
  g_last_error[0] = '\0';
  if (bytes == nullptr) return fail(FN_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  if (glu != 0 && glu != 1) return fail(FN_ERR_INVALID_ARG, "glu must be 0 or 1");
  fn_status st = check_int8_shape(M, d, N, glu != 0);
  if (st != FN_OK || M == 0) return st;
  int dev = 0;
  const int sms = device_sm_count(&dev);
  if (sms <= 1) return fail(FN_ERR_CUDA, "cannot query the current device");
  *bytes = int8_workspace(M, d, glu ? 2 * N : N, sms).bytes;
  return FN_OK;
}

fn_status flashnorm_linear_int8(const void* x, const void* Q, const void* scales, void* y, int64_t M, int64_t d, int64_t N,
                                float eps, int norm, int out_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  g_last_error[0] = '\0';
  return run_int8(x, Q, scales, y, M, d, N, eps, norm, out_dtype, false, workspace, workspace_bytes,
                  static_cast<cudaStream_t>(stream));
}

fn_status flashnorm_glu_int8(const void* x, const void* Q, const void* scales, void* y, int64_t M, int64_t d, int64_t F,
                             float eps, int out_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  g_last_error[0] = '\0';
  return run_int8(x, Q, scales, y, M, d, F, eps, 1, out_dtype, true, workspace, workspace_bytes,
                  static_cast<cudaStream_t>(stream));
}

}  // extern "C"
