// cross_entropy_small.cuh — the vocabulary head's cross entropy for at most 32 rows, bound by the bytes of W*.
//
// Operands swapped as in decode_tc.cuh: 128 rows of W* form the MMA's M side, the tokens its N side, so that a slab's MMAs
// cost next to nothing and the kernel only streams W*, one persistent CTA per SM with a deep ring. An epilogue thread owns
// one vocabulary row of each slab and half of the tokens; it keeps a running (maximum, sum) per token over all slabs of its
// CTA. At the end the lanes of a warp join theirs (each exchange halves the tokens a lane holds), every CTA writes one pair
// per token, and the last CTA to arrive joins all of them in a fixed order. The pass before it takes 1/rms and zeroes the
// arrival counter; W* and x do not depend on it and are fetched meanwhile, so it reads nothing but x: its loads queue behind
// W*'s, and when it fetched the targets' rows of W* for their logits too, the epilogue waited for it (23 rows x 576 x
// 49152, call after call: 18.4 us, 17.7 so). The targets' logits (ce_row_dot) are taken by the epilogue warps before they wait
// for that pass, a row per CTA where there are enough CTAs.
//
// Bound: HBM. 23 x 576 x 49152: 16.8 us for 57 MB (8.7 at the copy rate): 4 to start, 3 a slab, 2.5 for the join (a warp per
// token instead of 8 lanes: 6.4). The CTA-pair product, which spends 256 rows of MMA on them, takes 19.5 and a join of 5.
//
// Sums over k are taken in chunks of 1024, as for the CTA-pair product (its accumulators drift the same way).
//
// Warps: 0 = TMA producer, 1 = TMEM allocator + MMA issuer, 2..9 = epilogue, two per lane quarter.
#pragma once

#include "cross_entropy.cuh"

namespace fn {

constexpr int kCsRows = 128;
constexpr int kCsStages = 8;
constexpr int kCsThreads = 320;
constexpr int kCsChunk = 16;  // stages per accumulation

__host__ __device__ constexpr int ce_small_smem_bytes(int tokens) {
  return 1024 + kCsStages * (kCsRows * 128 + tokens * 128) + 256 + tokens * 32;
}

struct CeSmallParams {
  const float* rstd;
  float* tlogit;      // [M] x . W*[target]
  const uint16_t* x;
  const uint16_t* W;
  const long long* targets;
  float2* part;       // [M][CTAs]
  unsigned* arrived;  // zeroed by the pass before
  float* loss;
  float* lse;
  int M, K, V, num_kb;
  long long ignore;
};

// NT: tokens per epilogue thread; the MMA has 2 NT.
template <int NT>
__global__ void __launch_bounds__(kCsThreads, 1)
    k_ce_small(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, CeSmallParams p) {
  constexpr int kTok = 2 * NT;
  constexpr int kWBytes = kCsRows * 128, kXBytes = kTok * 128;
  constexpr uint32_t kCols = kTok < 32 ? 32 : kTok;  // per accumulator
  constexpr int kJoin = 256 / kTok;                  // lanes per token in the final join
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* sW = smem;
  uint8_t* sX = sW + kCsStages * kWBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sX + kCsStages * kXBytes);
  uint64_t* empty = full + kCsStages;
  uint64_t* acc_full = empty + kCsStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2]
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile unsigned* arrival = reinterpret_cast<volatile unsigned*>(tmem_slot + 2);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int slabs = (p.V + kCsRows - 1) / kCsRows;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kCsStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 2 * kCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int s = 0, issued = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int slab = static_cast<int>(blockIdx.x); slab < slabs && ok; slab += static_cast<int>(gridDim.x)) {
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], kWBytes + kXBytes);
          tma_load_2d(sW + s * kWBytes, &tm_w, &full[s], kb * 64, slab * kCsRows);
          tma_load_2d(sX + s * kXBytes, &tm_x, &full[s], kb * 64, 0);
          ++issued;
          if (++s == kCsStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      grid_dep_launch();
      if (ok) {
        // no arrival on this CTA's barriers (an MMA commit completes asynchronously) may be in flight at its exit
        for (int i = 0; i < kCsStages; ++i) {
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag)) break;
          if (++s == kCsStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      } else {
        const int pending = issued < kCsStages ? issued : kCsStages;
        for (int i = 1; i <= pending; ++i) {
          int st = s - i;
          uint32_t pp = ph;
          if (st < 0) {
            st += kCsStages;
            pp ^= 1u;
          }
          const unsigned long long t0 = globaltimer_ns();
          while (!mbar_try_wait(&full[st], pp) && globaltimer_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = make_idesc_bf16(kCsRows, kTok);
      const uint64_t dw0 = make_sdesc_sw128(smem_u32(sW)), dx0 = make_sdesc_sw128(smem_u32(sX));
      int s = 0, acc = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool ok = true;
      for (int slab = static_cast<int>(blockIdx.x); slab < slabs && ok; slab += static_cast<int>(gridDim.x)) {
        for (int kb = 0; kb < p.num_kb && ok;) {
          const int end = min(kb + kCsChunk, p.num_kb);
          if (!mbar_wait(&acc_empty[acc], acc_ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc) * kCols;
          for (int first = kb; kb < end; ++kb) {
            if (!mbar_wait(&full[s], ph, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint64_t dw = dw0 + static_cast<uint64_t>(s * (kWBytes / 16)), dx = dx0 + static_cast<uint64_t>(s * (kXBytes / 16));
#pragma unroll
            for (int k = 0; k < 4; ++k) tc_mma_bf16(d_tmem, dw + 2 * k, dx + 2 * k, idesc, kb != first || k != 0 ? 1u : 0u);
            tc_commit(&empty[s]);
            if (++s == kCsStages) {
              s = 0;
              ph ^= 1u;
            }
          }
          if (!ok) break;
          tc_commit(&acc_full[acc]);
          acc ^= 1;
          if (acc == 0) acc_ph ^= 1u;
        }
      }
      if (!ok) {
        tc_commit(drain);
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int w = warp - 2, q = warp & 3, half = w >> 2;
    for (int row = static_cast<int>(blockIdx.x) + w * static_cast<int>(gridDim.x); row < p.M; row += 8 * static_cast<int>(gridDim.x)) {
      const long long t = __ldcg(p.targets + row);
      if (!target_is_class(t, p.V)) continue;
      const float zt = ce_row_dot(p.x + static_cast<size_t>(row) * p.K, p.W + static_cast<size_t>(t) * p.K, p.K, lane);
      if (lane == 0) p.tlogit[row] = zt;
    }
    grid_dep_wait();
    // lane j: the target of the warp's token j
    const long long target = lane < NT && half * NT + lane < p.M ? __ldg(p.targets + half * NT + lane) : -1;
    float r2[NT], m[NT], s[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int t = half * NT + j;
      r2[j] = t < p.M ? __ldcg(p.rstd + t) * kLog2e : 0.f;
      m[j] = -1e38f;  // finite: a logit of -inf then adds 2^(-inf) = 0, not NaN
      s[j] = 0.f;
    }
    int acc = 0;
    uint32_t acc_ph = 0;
    bool ok = true;
    for (int slab = static_cast<int>(blockIdx.x); slab < slabs && ok; slab += static_cast<int>(gridDim.x)) {
      float z[NT];
      for (int kb = 0; kb < p.num_kb; kb += kCsChunk) {
        if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[acc], acc_ph, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t at = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc) * kCols + half * NT;
        uint32_t v[NT / 8][8];
#pragma unroll
        for (int b = 0; b < NT / 8; ++b) tmem_ld8(at + 8 * b, v[b]);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          asm volatile("" : "+r"(v[j >> 3][j & 7]));
          z[j] = (kb == 0 ? 0.f : z[j]) + __uint_as_float(v[j >> 3][j & 7]);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[acc]);
        acc ^= 1;
        if (acc == 0) acc_ph ^= 1u;
      }
      const long long row = target - (static_cast<long long>(slab) * kCsRows + q * 32);
      unsigned mine = 0;  // tokens whose target is this row: their logits join at the end
      for (unsigned hits = __ballot_sync(0xffffffffu, ok && row >= 0 && row < 32); hits != 0; hits &= hits - 1) {
        const int j0 = __ffs(hits) - 1;
        if (__shfl_sync(0xffffffffu, static_cast<int>(row), j0) == lane) mine |= 1u << j0;
      }
      if (ok && slab * kCsRows + q * 32 + lane < p.V) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (mine >> j & 1u) continue;
          const float d = fmaf(z[j], r2[j], -m[j]);
          const float e = ex2(-fabsf(d));
          s[j] = d > 0.f ? fmaf(s[j], e, 1.0f) : s[j] + e;
          m[j] = d > 0.f ? z[j] * r2[j] : m[j];
        }
      }
    }
    // join over the lanes: an exchange with lane ^ o halves the tokens each holds; then tokens are lane / (32 / NT)
    auto join = [](float& am, float& as, float bm, float bs) {
      const float d = bm - am, e = ex2(-fabsf(d));
      as = d > 0.f ? fmaf(as, e, bs) : fmaf(bs, e, as);
      am = d > 0.f ? bm : am;
    };
    int o = 16;
#pragma unroll
    for (int n = NT / 2; n >= 1; n >>= 1, o >>= 1) {
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int j = 0; j < n; ++j) {
        const float bm = __shfl_xor_sync(0xffffffffu, up ? m[j] : m[j + n], o), bs = __shfl_xor_sync(0xffffffffu, up ? s[j] : s[j + n], o);
        m[j] = up ? m[j + n] : m[j];
        s[j] = up ? s[j + n] : s[j];
        join(m[j], s[j], bm, bs);
      }
    }
    for (; o >= 1; o >>= 1) join(m[0], s[0], __shfl_xor_sync(0xffffffffu, m[0], o), __shfl_xor_sync(0xffffffffu, s[0], o));
    // the four quarters' pairs through shared memory, then one per CTA and token
    float2* quarters = reinterpret_cast<float2*>(sX + kCsStages * kXBytes + 256);  // [4][kTok]
    if (lane % (32 / NT) == 0)
      quarters[q * kTok + half * NT + lane / (32 / NT)] =
          make_float2(m[0], *abort_flag || !ok ? __int_as_float(0x7fc00000) : s[0]);  // the status word reports a timeout
    named_bar_sync(1, 256);
    const int parts = static_cast<int>(gridDim.x), tok = static_cast<int>(threadIdx.x) - 64;
    if (tok < p.M) {
      float2 a = quarters[tok];
#pragma unroll
      for (int k = 1; k < 4; ++k) join(a.x, a.y, quarters[k * kTok + tok].x, quarters[k * kTok + tok].y);
      __stcg(p.part + static_cast<size_t>(tok) * parts + blockIdx.x, a);
    }
    named_bar_sync(1, 256);  // the CTA's pairs come before its arrival (barrier, then release)
    if (threadIdx.x == 64) *arrival = atom_add_acq_rel_gpu(p.arrived, 1u);
    named_bar_sync(1, 256);
    if (*arrival == gridDim.x - 1) {
      const int row = tok / kJoin;
      const bool live = row < p.M;
      // the logit is not written, nor used, where the target is no class
      const float zt = live ? __ldcg(p.tlogit + row) : 0.f, rstd = live ? __ldcg(p.rstd + row) : 0.f;
      const long long t = live ? __ldcg(p.targets + row) : p.ignore;
      // all tokens at once, 19 pairs of each lane in flight: every other SM is idle meanwhile
      ce_join_row<kJoin, 19>(p.part, parts, rstd, zt, t, p.loss, p.lse, row, live, p.V, p.ignore, lane);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem_base, 2 * kCols);
}

}  // namespace fn
