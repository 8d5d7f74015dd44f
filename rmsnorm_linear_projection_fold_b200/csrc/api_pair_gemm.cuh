// api_pair_gemm.cuh — tile plan and launch of the CTA-pair matrix product (pair_gemm.cuh). Part of flashnorm.cu.
#pragma once

namespace {

// Tile width by choose_bn's cost (waves of tiles over the CTA pairs, times the width plus a fixed cost), row tiles
// in bands of eight: the pairs running at once then read 8 row tiles and about 9 column tiles of the operands.
void plan_pair_gemm(fn::PairGemmParams* p, int64_t M, int64_t N, int64_t num_kb, int sms, int step, int ksplit) {
  p->M = static_cast<int>(M);
  p->N = static_cast<int>(N);
  p->num_kb = static_cast<int>(num_kb);
  p->bn = choose_bn((M + 1) / 2, N, sms / 2, step);
  p->num_m_tiles = static_cast<int>((M + 255) / 256);
  p->num_n_tiles = static_cast<int>((N + p->bn - 1) / p->bn);
  p->band = std::min(8, p->num_m_tiles);
  p->ksplit = ksplit;
  p->early = fn::PG_EARLY_NONE;
  p->live_is_k = 0;
  p->live = nullptr;
}

template <int KIND, bool A_MN, bool B_MN, class Epi>
fn_status launch_pair_gemm(const CUtensorMap& ta, const CUtensorMap& tb, const fn::PairGemmParams& p,
                           const typename Epi::Params& ep, int sms, int dev, cudaStream_t s, const char* what) {
  auto kern = fn::k_pair_gemm<KIND, A_MN, B_MN, Epi>;
  constexpr int smem = fn::pair_gemm_smem_bytes();
  static bool configured[kMaxDevices] = {false};
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_fail(e, what);
    configured[dev] = true;
  }
  const int64_t items = static_cast<int64_t>(p.num_m_tiles) * p.num_n_tiles * p.ksplit;
  if (items > kMaxDim) return fail(FN_ERR_UNSUPPORTED, "%s: too many tiles", what);
  const int pairs = static_cast<int>(std::min<int64_t>(items, sms / 2));
  cudaError_t e = launch_kernel(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(fn::kPgThreads), smem, s, 2, ta, tb, p, ep);
  if (e != cudaSuccess) return cuda_fail(e, what);
  return FN_OK;
}

}  // namespace
