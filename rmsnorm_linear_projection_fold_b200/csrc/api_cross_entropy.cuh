// api_cross_entropy.cuh — host side of the vocabulary head's cross entropy and its gradient (cross_entropy.cuh). Part of
// flashnorm.cu.
#pragma once

namespace {

// 2-D bf16 operand stored MN-major, [k][cols] with row stride ld: 64 cols x 64 k boxes, 128-byte swizzle.
fn_status make_mn_map(CUtensorMap* map, const void* ptr, int64_t cols, int64_t k, int64_t ld) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(k)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[2] = {64u, 64u};
  CUresult r = encode_cached(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (r == CUDA_ERROR_NOT_FOUND) return fail(FN_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  if (r != CUDA_SUCCESS) return fail(FN_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", static_cast<int>(r));
  return FN_OK;
}

// The same as blocks of 64 columns, cols % 64 == 0: boxes of `blocks` blocks x 64 k, one copy per stage.
fn_status make_mn_block_map(CUtensorMap* map, const void* ptr, int64_t cols, int64_t k, int64_t ld, int blocks) {
  cuuint64_t dims[3] = {64u, static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(cols / 64)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, 128u};
  cuuint32_t box[3] = {64u, 64u, static_cast<cuuint32_t>(blocks)};
  CUresult r = encode_cached(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (r == CUDA_ERROR_NOT_FOUND) return fail(FN_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  if (r != CUDA_SUCCESS) return fail(FN_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", static_cast<int>(r));
  return FN_OK;
}

fn_status make_mn_operand(CUtensorMap* map, fn::PairGemmParams* p, const void* ptr, int64_t cols, int64_t k) {
  p->b_blocks = cols % 64 == 0;
  return p->b_blocks ? make_mn_block_map(map, ptr, cols, k, cols, p->bn / 128) : make_mn_map(map, ptr, cols, k, cols);
}

// 2-D bf16 K-major operand [rows][k] with row stride ld: 64 k x box_rows boxes, 128-byte swizzle.
fn_status make_k_map(CUtensorMap* map, const void* ptr, int64_t k, int64_t rows, int64_t ld, int box_rows) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(box_rows)};
  CUresult r = encode_cached(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (r == CUDA_ERROR_NOT_FOUND) return fail(FN_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  if (r != CUDA_SUCCESS) return fail(FN_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", static_cast<int>(r));
  return FN_OK;
}

// Masks of 32 live rows, whole row tiles of the logits' product.
int64_t ce_ld_hits(int64_t M) { return round_up(M, 256) / 32; }

// What a call works through and where the parts of its workspace start.
struct CePlan {
  int64_t piece;   // vocabulary columns of a piece (forward: all)
  int64_t pieces;
  int n_tiles;     // column tiles of a full piece
  int ksplit;      // K ranges of dx's product, and of dW*'s where it goes through planes
  int dw_ksplit;
  int64_t arrived, failed, rstd, part, tlogit;       // forward (arrived, tlogit: few rows; failed: more)
  int64_t n_live, rows, rank_of, target, u, ct, hits, xc, P, acc, dw_acc, bytes;  // backward (and part)
};

// Stages per accumulation of the forward's logits: 1024 k. At k = 4096 the loss is then 3.4e-7 off (relative), 1.5e-6 with one
// sum over all k; each accumulation of a tile costs about 650 cycles (2048 x 4096 x 32000: 376 against 361 us).
constexpr int kCeFwdChunk = 16;

// Tile width of the products whose B is MN-major (x or W*, [k][d]).
int ce_mn_width(int64_t d) { return d > 128 ? 256 : 128; }

// Up to so many classes, and with a row for every sixteenth at least, dW* is finished by a pass of its own (k_ce_dw), its
// product cut into K ranges. With few rows the pass costs more than it saves (5 x 1080 x 1843: 9 us).
constexpr int64_t kCeSmallVocab = 2048;

// What an item of so many stages takes, in stages: at least its epilogue. With 6, 12 and 24 of them the gradient of 517 x 576 x
// 50257 takes 133, 125 and 146 us, of 60 x 1024 x 50000 97, 102 and 130, of 128 x 4096 x 32000 229, 217 and 266, of 300 x 2048 x
// 32000 195 to 220, 192 and 179.
int64_t ce_item_cost(int64_t kb) { return std::max<int64_t>(kb, 12); }

// K ranges of a product that shares a launch with another: few enough planes, many enough items that the longest share of
// any pair fits into an even part of both products' work.
int ce_ksplit(const fn::PairGemmParams& g, const fn::PairGemmParams& other, int pairs) {
  const int64_t items = static_cast<int64_t>(g.num_m_tiles) * g.num_n_tiles;
  const int64_t all = items * ce_item_cost(g.num_kb) + static_cast<int64_t>(other.num_m_tiles) * other.num_n_tiles * ce_item_cost(other.num_kb);
  const int64_t even = (all + pairs - 1) / pairs;
  int k = 1;
  while (k < 64 && g.num_kb / (k + 1) >= 8 &&
         (items * k + pairs - 1) / pairs * ce_item_cost((g.num_kb + k - 1) / k) > even)
    ++k;
  return k;
}

// Items of job 1 that take as long as one of job 0.
int ce_extra(const fn::PairGemmParams& p, const fn::PairGemmParams& q) {
  return static_cast<int>(std::max<int64_t>(1, ce_item_cost(p.num_kb / p.ksplit) / ce_item_cost(q.num_kb / q.ksplit)));
}

// Up to so many rows the loss streams W* past the tokens (cross_entropy_small.cuh). Call after call, so and on CTA pairs:
//   576 x 49152    1 row 15.8 and 24.6 us, 16 rows 17.2 and 22.1, 32 rows 19.2 and 22.6 (64 rows: 27.3 and 22.9, the tokens' tile
//                  being fetched with every stage)
//   4096 x 32000   1 row 48.7 and 76.4, 16 rows 50.1 and 56.1, 32 rows 52.8 and 56.6
//   1024 x 128256  1 row 47.8 and 73.2, 16 rows 49.2 and 71.2, 32 rows 52.2 and 67.4
constexpr int kCeSmallRows = 32;
constexpr int kCeFwdParts = fn::CeFwdEpi<false>::kParts;

// P of a piece: at most so many bytes, unless that were fewer than kCePieceMin columns, between which dx's sums (8 bytes read
// and written per element) would weigh too much. With half the bytes, so, and with room for all of P the gradient takes 1.28,
// 1.23 and 1.20 ms at 2048 x 4096 x 32000, 2.92, 2.66 and 2.56 at 4096 x 2048 x 65536 (512 MB), 0.89, 0.79 and 0.67 to 0.73 at
// 4096 x 576 x 49152: memory against time.
constexpr int64_t kCePieceBytes = int64_t{64} << 20, kCePieceMin = 4096;

CePlan ce_plan(int64_t M, int64_t d, int64_t V, bool backward, int sms) {
  CePlan c = {};
  c.piece = V, c.pieces = 1, c.ksplit = 1;
  if (backward) {
    const int64_t cap = std::max<int64_t>(kCePieceMin, kCePieceBytes / (2 * M) / 256 * 256);
    c.pieces = (V + cap - 1) / cap;
    c.piece = c.pieces == 1 ? V : round_up((V + c.pieces - 1) / c.pieces, 256);
    c.pieces = (V + c.piece - 1) / c.piece;
  }
  fn::PairGemmParams g;
  plan_pair_gemm(&g, M, c.piece, (d + 63) / 64, sms, 32);
  c.n_tiles = g.num_n_tiles;
  if (!backward) {
    c.arrived = c.failed = 0;
    c.rstd = 256;
    c.part = c.rstd + round_up(4 * M, 256);
    if (M <= kCeSmallRows) {
      c.tlogit = c.part + round_up(8ll * sms * M, 256);
      c.bytes = c.tlogit + round_up(4 * M, 256);
      return c;
    }
    c.bytes = c.part + round_up(8ll * kCeFwdParts * c.n_tiles * M, 256);
    return c;
  }
  fn::PairGemmParams w;
  plan_pair_gemm_bn(&g, M, d, (c.piece + 63) / 64, ce_mn_width(d), 1);
  plan_pair_gemm_bn(&w, c.piece, d, (M + 63) / 64, ce_mn_width(d), 1);
  c.ksplit = ce_ksplit(g, w, sms / 2);
  c.dw_ksplit = V <= kCeSmallVocab && 16 * M >= V ? ce_ksplit(w, g, sms / 2) : 0;
  const int64_t Mp = round_up(M, 64);  // the packed rows, zeros at their end
  c.n_live = 0;
  c.rows = 256;
  c.rank_of = c.rows + round_up(16 * M, 256);
  c.target = c.rank_of + round_up(4 * M, 256);
  c.u = c.target + round_up(4 * M, 256);
  c.ct = c.u + round_up(4 * M, 256);
  c.hits = c.ct + round_up(4 * M, 256);
  c.part = c.hits + round_up(4 * ((c.piece + 31) / 32) * ce_ld_hits(M), 256);
  c.xc = c.part + round_up(4ll * fn::CeGradEpi::kParts * c.n_tiles * c.pieces * M, 256);
  c.P = c.xc + round_up(2 * Mp * d, 256);
  c.acc = c.P + 2 * Mp * round_up(c.piece, 64);
  c.dw_acc = c.acc + round_up(4 * c.ksplit * M * d, 256);
  c.bytes = c.dw_acc + 4 * c.dw_ksplit * c.piece * d;
  return c;
}

fn_status check_ce_shape(int64_t M, int64_t d, int64_t V) {
  if (M < 0 || M > kMaxDim / 2) return fail(FN_ERR_INVALID_ARG, "M = %lld out of range", (long long)M);
  if (d < 8 || d > kMaxDim || d % 8 != 0) return fail(FN_ERR_INVALID_ARG, "d = %lld must be a positive multiple of 8", (long long)d);
  if (V < 1 || V > kMaxDim / 2) return fail(FN_ERR_INVALID_ARG, "V = %lld out of range", (long long)V);
  return FN_OK;
}

fn_status check_ce_call(const void* x, const void* w, const void* targets, const void* a, const char* an, const void* b,
                        const char* bn, float eps, const void* workspace, int64_t workspace_bytes) {
  fn_status st;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(FN_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (workspace_bytes < 0) return fail(FN_ERR_INVALID_ARG, "workspace_bytes < 0");
  if ((st = check_ptr(x, "x")) != FN_OK) return st;
  if ((st = check_ptr(w, "W*")) != FN_OK) return st;
  if ((st = check_vec(targets, "targets", 8)) != FN_OK) return st;
  if ((st = check_vec(a, an, 4)) != FN_OK) return st;
  if ((st = check_vec(b, bn, 4)) != FN_OK) return st;
  return check_ptr(workspace, "workspace");
}

fn_status launch_rstd(const void* x, float* rstd, unsigned* zero, int64_t M, int64_t d, float eps, cudaStream_t s) {
  cudaError_t e = launch_kernel(fn::k_row_rstd, dim3(static_cast<unsigned>((M + 7) / 8)), dim3(256), 0, s, 1,
                                static_cast<const uint16_t*>(x), rstd, zero, static_cast<int>(M), static_cast<int>(d), eps);
  return e == cudaSuccess ? FN_OK : cuda_fail(e, "row statistics launch");
}

template <int NT>
fn_status launch_ce_small(const CUtensorMap& tw, const CUtensorMap& tx, const fn::CeSmallParams& p, int sms, int dev,
                          cudaStream_t s) {
  auto kern = fn::k_ce_small<NT>;
  constexpr int smem = fn::ce_small_smem_bytes(2 * NT);
  static bool configured[kMaxDevices] = {false};
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute (cross entropy, few rows)");
    configured[dev] = true;
  }
  const int slabs = (p.V + fn::kCsRows - 1) / fn::kCsRows;
  cudaError_t e = launch_kernel(kern, dim3(static_cast<unsigned>(std::min(slabs, sms))), dim3(fn::kCsThreads), smem, s, 1, tw, tx, p);
  return e == cudaSuccess ? FN_OK : cuda_fail(e, "cross entropy launch (few rows)");
}

}  // namespace

extern "C" {

fn_status flashnorm_cross_entropy_workspace_bytes(int64_t M, int64_t d, int64_t V, int backward, int64_t* bytes) {
  g_last_error[0] = '\0';
  if (bytes == nullptr) return fail(FN_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  if (backward != 0 && backward != 1) return fail(FN_ERR_INVALID_ARG, "backward must be 0 or 1");
  fn_status st = check_ce_shape(M, d, V);
  if (st != FN_OK || M == 0) return st;
  int dev = 0;
  const int sms = device_sm_count(&dev);
  if (sms <= 1) return fail(FN_ERR_CUDA, "cannot query the current device");
  *bytes = ce_plan(M, d, V, backward != 0, sms).bytes;
  return FN_OK;
}

fn_status flashnorm_linear_cross_entropy(const void* x, const void* Wstar, const void* targets, void* loss, void* lse,
                                         int64_t M, int64_t d, int64_t V, float eps, int64_t ignore_index,
                                         void* workspace, int64_t workspace_bytes, void* stream) {
  g_last_error[0] = '\0';
  fn_status st = check_ce_shape(M, d, V);
  if (st != FN_OK || M == 0) return st;
  if ((st = check_ce_call(x, Wstar, targets, loss, "loss", lse, "lse", eps, workspace, workspace_bytes)) != FN_OK) return st;
  int dev = 0;
  const int sms = device_sm_count(&dev);
  if (sms <= 1) return fail(FN_ERR_CUDA, "cannot query the current device");
  const CePlan c = ce_plan(M, d, V, false, sms);
  if (workspace_bytes < c.bytes)
    return fail(FN_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)c.bytes);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  float* rstd = reinterpret_cast<float*>(base + c.rstd);
  if (M <= kCeSmallRows) {
    fn::CeSmallParams p;
    p.rstd = rstd;
    p.tlogit = reinterpret_cast<float*>(base + c.tlogit);
    p.targets = static_cast<const long long*>(targets);
    p.part = reinterpret_cast<float2*>(base + c.part);
    p.arrived = reinterpret_cast<unsigned*>(base + c.arrived);
    p.loss = static_cast<float*>(loss);
    p.lse = static_cast<float*>(lse);
    p.x = static_cast<const uint16_t*>(x);
    p.W = static_cast<const uint16_t*>(Wstar);
    p.M = static_cast<int>(M);
    p.K = static_cast<int>(d);
    p.V = static_cast<int>(V);
    p.num_kb = static_cast<int>((d + 63) / 64);
    p.ignore = ignore_index;
    const int tokens = M <= 16 ? 16 : kCeSmallRows;
    CUtensorMap tx, tw;
    if ((st = make_k_map(&tx, x, d, M, d, tokens)) != FN_OK) return st;
    if ((st = make_k_map(&tw, Wstar, d, V, d, fn::kCsRows)) != FN_OK) return st;
    if ((st = launch_rstd(x, rstd, p.arrived, M, d, eps, s)) != FN_OK) return st;
    return tokens == 16 ? launch_ce_small<8>(tw, tx, p, sms, dev, s) : launch_ce_small<16>(tw, tx, p, sms, dev, s);
  }
  fn::CeFwdParams ep;
  ep.rstd = rstd;
  ep.targets = static_cast<const long long*>(targets);
  ep.part = reinterpret_cast<float2*>(base + c.part);
  fn::PairGemmParams p;
  plan_pair_gemm(&p, M, V, (d + 63) / 64, sms, 32);
  p.kchunk = kCeFwdChunk;
  p.early = fn::PG_EARLY_AB;  // neither operand depends on the row statistics
  p.failed = reinterpret_cast<unsigned*>(base + c.failed);
  CUtensorMap tx, tw;
  if ((st = make_k_map(&tx, x, d, M, d, 128)) != FN_OK) return st;
  if ((st = make_k_map(&tw, Wstar, d, V, d, p.bn / 2)) != FN_OK) return st;
  if ((st = launch_rstd(x, rstd, p.failed, M, d, eps, s)) != FN_OK) return st;
  const char* what = "cross entropy GEMM";
  st = p.num_kb > kCeFwdChunk
           ? launch_pair_gemm<fn::PG_BF16, fn::PgJob<false, false, fn::CeFwdEpi<true>>>(tx, tw, p, ep, sms, dev, s, what)
           : launch_pair_gemm<fn::PG_BF16, fn::PgJob<false, false, fn::CeFwdEpi<false>>>(tx, tw, p, ep, sms, dev, s, what);
  if (st != FN_OK) return st;
  cudaError_t e = launch_kernel(fn::k_ce_join, dim3(static_cast<unsigned>((M + 7) / 8)), dim3(256), 0, s, 1,
                                static_cast<const float2*>(ep.part), ep.rstd, static_cast<const uint16_t*>(x),
                                static_cast<const uint16_t*>(Wstar), ep.targets, static_cast<const unsigned*>(p.failed),
                                static_cast<float*>(loss), static_cast<float*>(lse), p.M, static_cast<int>(d), p.N, kCeFwdParts * p.num_n_tiles,
                                static_cast<long long>(ignore_index));
  return e == cudaSuccess ? FN_OK : cuda_fail(e, "cross entropy join launch");
}

fn_status flashnorm_linear_cross_entropy_backward(const void* g, const void* x, const void* Wstar, const void* targets,
                                                  const void* lse, void* dx, void* dWstar, int64_t M, int64_t d,
                                                  int64_t V, float eps, int64_t ignore_index, void* workspace,
                                                  int64_t workspace_bytes, void* stream) {
  g_last_error[0] = '\0';
  fn_status st = check_ce_shape(M, d, V);
  if (st != FN_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {  // no rows: the weight's gradient is zero
    if ((st = check_ptr(dWstar, "dW*")) != FN_OK) return st;
    cudaError_t e = cudaMemsetAsync(dWstar, 0, static_cast<size_t>(V) * static_cast<size_t>(d) * 2, s);
    return e == cudaSuccess ? FN_OK : cuda_fail(e, "clearing dW*");
  }
  if ((st = check_ce_call(x, Wstar, targets, g, "g", lse, "lse", eps, workspace, workspace_bytes)) != FN_OK) return st;
  if ((st = check_ptr(dx, "dx")) != FN_OK) return st;
  if ((st = check_ptr(dWstar, "dW*")) != FN_OK) return st;
  int dev = 0;
  const int sms = device_sm_count(&dev);
  if (sms <= 1) return fail(FN_ERR_CUDA, "cannot query the current device");
  const CePlan c = ce_plan(M, d, V, true, sms);
  if (workspace_bytes < c.bytes)
    return fail(FN_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)c.bytes);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  int* n_live = reinterpret_cast<int*>(base + c.n_live);
  fn::CeRow* rows = reinterpret_cast<fn::CeRow*>(base + c.rows);
  int* rank_of = reinterpret_cast<int*>(base + c.rank_of);
  uint16_t* xc = reinterpret_cast<uint16_t*>(base + c.xc);
  const fn::CeLive live = {n_live, reinterpret_cast<int*>(base + c.target), reinterpret_cast<float*>(base + c.u),
                          reinterpret_cast<unsigned*>(base + c.hits), static_cast<int>(ce_ld_hits(M))};
  float* ct = reinterpret_cast<float*>(base + c.ct);
  float* cpart = reinterpret_cast<float*>(base + c.part);
  uint16_t* P = reinterpret_cast<uint16_t*>(base + c.P);
  float* acc = reinterpret_cast<float*>(base + c.acc);
  const int64_t ldp = round_up(c.piece, 64), Mp = round_up(M, 64);
  // about 256 blocks at most: each counts the live rows before its own
  const int64_t per_block = round_up((M + 255) / 256, 8);
  cudaError_t e = launch_kernel(fn::k_ce_pack, dim3(static_cast<unsigned>((M + per_block - 1) / per_block)), dim3(256), 0, s, 1,
                                static_cast<const uint16_t*>(x), static_cast<const long long*>(targets),
                                static_cast<const float*>(lse), static_cast<const float*>(g),
                                static_cast<const uint16_t*>(Wstar), xc, rows, live.target, live.u, ct, rank_of, n_live,
                                static_cast<int>(M), static_cast<int>(d), static_cast<int>(V),
                                static_cast<int>(per_block), eps, static_cast<long long>(ignore_index));
  if (e != cudaSuccess) return cuda_fail(e, "cross entropy pack launch");
  int parts = 0;
  for (int64_t v0 = 0; v0 < V; v0 += c.piece) {
    const int64_t width = std::min(c.piece, V - v0);
    const uint16_t* W = static_cast<const uint16_t*>(Wstar) + v0 * d;
    CUtensorMap ta, tb, ta1, tb1;
    // the logits again, and P from them
    fn::PairGemmParams p, q;
    plan_pair_gemm(&p, M, c.piece, (d + 63) / 64, sms, 32);
    p.N = static_cast<int>(width);
    p.num_n_tiles = static_cast<int>((width + p.bn - 1) / p.bn);
    p.live = n_live;
    const fn::CeGradParams ge = {rows, P, cpart + static_cast<int64_t>(parts) * M, static_cast<int>(ldp), static_cast<int>(v0),
                                 V > kCeSmallVocab ? 3 : 33, live};
    parts += fn::CeGradEpi::kParts * p.num_n_tiles;
    if ((st = make_k_map(&ta, xc, d, Mp, d, 128)) != FN_OK) return st;
    if ((st = make_k_map(&tb, W, d, width, d, p.bn / 2)) != FN_OK) return st;
    if ((st = launch_pair_gemm<fn::PG_BF16, fn::PgJob<false, false, fn::CeGradEpi>>(ta, tb, p, ge, sms, dev, s, "cross entropy P")) != FN_OK)
      return st;
    // dx += P W* and dW* = P^T x
    plan_pair_gemm_bn(&p, M, d, (width + 63) / 64, ce_mn_width(d), c.ksplit);
    p.live = n_live;
    const fn::CeDxParams xe = {acc, static_cast<int>(d), v0 > 0};
    if ((st = make_k_map(&ta, P, width, Mp, ldp, 128)) != FN_OK) return st;
    if ((st = make_mn_operand(&tb, &p, W, d, width)) != FN_OK) return st;
    plan_pair_gemm_bn(&q, width, d, (M + 63) / 64, ce_mn_width(d), 1);
    q.live = n_live;
    q.live_is_k = 1;
    if ((st = make_mn_block_map(&ta1, P, ldp, Mp, ldp, 2)) != FN_OK) return st;
    if ((st = make_mn_operand(&tb1, &q, xc, d, Mp)) != FN_OK) return st;
    uint16_t* dWp = static_cast<uint16_t*>(dWstar) + v0 * d;
    const char* what = "cross entropy gradients";
    using Dx = fn::PgJob<false, true, fn::CeDxEpi>;
    if (c.dw_ksplit) {
      q.ksplit = c.dw_ksplit;
      q.extra = ce_extra(p, q);
      float* planes = reinterpret_cast<float*>(base + c.dw_acc);
      const fn::CeDxParams we = {planes, static_cast<int>(d), 0};
      st = launch_pair_gemm2<Dx, fn::PgJob<true, true, fn::CeDxEpi>>(ta, tb, p, xe, ta1, tb1, q, we, sms, dev, s, what);
      if (st != FN_OK) return st;
      e = launch_kernel(fn::k_ce_dw, dim3(static_cast<unsigned>(width)), dim3(256), 0, s, 1, static_cast<const float*>(planes), live,
                        static_cast<const uint16_t*>(xc), dWp, static_cast<int>(width), static_cast<int>(d), c.dw_ksplit,
                        static_cast<int>(v0));
      if (e != cudaSuccess) return cuda_fail(e, "cross entropy dW launch");
    } else {
      q.extra = ce_extra(p, q);
      const fn::CeDwParams we = {live, xc, dWp, static_cast<int>(d), static_cast<int>(v0)};
      st = launch_pair_gemm2<Dx, fn::PgJob<true, true, fn::CeDwEpi>>(ta, tb, p, xe, ta1, tb1, q, we, sms, dev, s, what);
      if (st != FN_OK) return st;
    }
  }
  const bool narrow = d / 8 * c.ksplit + parts <= 128;  // loads of a row: a warp for it, else a block
  e = launch_kernel(narrow ? fn::k_ce_dx<32> : fn::k_ce_dx<256>, dim3(static_cast<unsigned>(narrow ? (M + 7) / 8 : M)), dim3(256), 0, s,
                    1, static_cast<const float*>(acc), static_cast<const float*>(cpart), static_cast<const fn::CeRow*>(rows),
                    static_cast<const float*>(live.u), static_cast<const float*>(ct), static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(Wstar),
                    static_cast<const int*>(rank_of), static_cast<uint16_t*>(dx), static_cast<int>(M), static_cast<int>(d),
                    c.ksplit, parts);
  return e == cudaSuccess ? FN_OK : cuda_fail(e, "cross entropy dx launch");
}

}  // extern "C"
