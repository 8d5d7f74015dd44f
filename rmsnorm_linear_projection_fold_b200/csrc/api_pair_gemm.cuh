// api_pair_gemm.cuh — tile plan and launch of the CTA-pair matrix product (pair_gemm.cuh). Part of flashnorm.cu.
#pragma once

namespace {

// Row tiles go in bands of eight: the pairs running at once then read 8 row tiles and about 9 column tiles of the
// operands.
void plan_pair_gemm_bn(fn::PairGemmParams* p, int64_t M, int64_t N, int64_t num_kb, int bn, int ksplit) {
  *p = {};
  p->M = static_cast<int>(M);
  p->N = static_cast<int>(N);
  p->num_kb = p->kchunk = static_cast<int>(num_kb);
  p->bn = bn;
  p->num_m_tiles = static_cast<int>((M + 255) / 256);
  p->num_n_tiles = static_cast<int>((N + bn - 1) / bn);
  p->band = std::min(8, p->num_m_tiles);
  p->ksplit = ksplit;
}

// Tile width by choose_bn's cost (waves of tiles over the CTA pairs, times the width plus a fixed cost).
void plan_pair_gemm(fn::PairGemmParams* p, int64_t M, int64_t N, int64_t num_kb, int sms, int step) {
  plan_pair_gemm_bn(p, M, N, num_kb, choose_bn((M + 1) / 2, N, sms / 2, step), 1);
}

int64_t pair_items(const fn::PairGemmParams& p) { return static_cast<int64_t>(p.num_m_tiles) * p.num_n_tiles * p.ksplit; }

template <typename Kern>
fn_status configure_pair_gemm(Kern kern, int parts, bool* configured, const char* what) {
  if (*configured) return FN_OK;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, fn::pair_gemm_smem_bytes(parts));
  if (e != cudaSuccess) return cuda_fail(e, what);
  *configured = true;
  return FN_OK;
}

template <int KIND, class J>
fn_status launch_pair_gemm(const CUtensorMap& ta, const CUtensorMap& tb, const fn::PairGemmParams& p,
                           const typename J::Params& ep, int sms, int dev, cudaStream_t s, const char* what) {
  auto kern = fn::k_pair_gemm<KIND, J>;
  constexpr int parts = J::Epi::kParts;
  static bool configured[kMaxDevices] = {false};
  fn_status st = configure_pair_gemm(kern, parts, &configured[dev], what);
  if (st != FN_OK) return st;
  const int64_t items = pair_items(p);
  if (items > kMaxDim) return fail(FN_ERR_UNSUPPORTED, "%s: too many tiles", what);
  const int pairs = static_cast<int>(std::min<int64_t>(items, sms / 2));
  cudaError_t e = launch_kernel(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(fn::pair_gemm_threads(parts)),
                                fn::pair_gemm_smem_bytes(parts), s, 2, ta, tb, p, ep);
  return e == cudaSuccess ? FN_OK : cuda_fail(e, what);
}

template <class J0, class J1>
fn_status launch_pair_gemm2(const CUtensorMap& ta0, const CUtensorMap& tb0, const fn::PairGemmParams& p0,
                            const typename J0::Params& ep0, const CUtensorMap& ta1, const CUtensorMap& tb1,
                            const fn::PairGemmParams& p1, const typename J1::Params& ep1, int sms, int dev,
                            cudaStream_t s, const char* what) {
  auto kern = fn::k_pair_gemm2<J0, J1>;
  constexpr int parts = J0::Epi::kParts;
  static bool configured[kMaxDevices] = {false};
  fn_status st = configure_pair_gemm(kern, parts, &configured[dev], what);
  if (st != FN_OK) return st;
  const int64_t items = pair_items(p0) + pair_items(p1);
  if (items > kMaxDim) return fail(FN_ERR_UNSUPPORTED, "%s: too many tiles", what);
  const int pairs = static_cast<int>(std::min<int64_t>(items, sms / 2));
  cudaError_t e = launch_kernel(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(fn::pair_gemm_threads(parts)),
                                fn::pair_gemm_smem_bytes(parts), s, 2, ta0, tb0, p0, ep0, ta1, tb1, p1, ep1);
  return e == cudaSuccess ? FN_OK : cuda_fail(e, what);
}

}  // namespace
