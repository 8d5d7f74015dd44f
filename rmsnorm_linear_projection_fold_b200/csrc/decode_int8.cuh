// decode_int8.cuh — the 8-bit integer projection for at most 16 rows (decode), bound by the bytes of Q, behind a row pass:
// for the shapes whose codes do not fit next to the ring of decode_int8_cluster.cuh.
//
// Operands swapped as in decode_tc.cuh: 128 rows of Q form the MMA's M side (kind::i8), the tokens its N side. The
// contraction of each 128-row slab is cut into K ranges over independent CTAs, two on every SM, so that small
// projections too keep the whole device loading; each writes its int32 partial sums to a workspace, and the last
// of a slab to arrive adds them (integer sums: the order cannot matter), scales and stores. The row pass before it
// has zeroed the slabs' arrival counters.
//
// Q does not depend on the row pass, so the first ring of Q stages is fetched while that pass still runs
// (programmatic launch): the row pass itself waits for everything before it, hence Q is in place by the time this
// kernel can start at all. Codes, rho and counters are touched only after griddepcontrol.wait.
//
// Warps: 0 = TMA producer, 1 = TMEM allocator + MMA issuer, 2..5 = epilogue.
#pragma once

#include "int8.cuh"

namespace fn {

constexpr int kI8Rows = 128;             // rows of Q per CTA (MMA M)
constexpr int kI8Tok = 16;               // token slots (MMA N)
constexpr int kI8WStage = kI8Rows * 128;  // 16 KB: 128 k
constexpr int kI8XStage = kI8Tok * 128;   // 2 KB
constexpr int kI8DecThreads = 192;
constexpr int kI8DecStages = 5;  // 90 KB: two CTAs per SM
constexpr unsigned kI8Gave = 1u << 16;  // added to a slab's counter by a CTA whose wait gave up

__host__ __device__ constexpr int decode_int8_smem_bytes() { return 1024 + kI8DecStages * (kI8WStage + kI8XStage) + 512; }

struct DecodeInt8Params {
  void* y;
  const float* rho;    // [M]
  const float* scale;  // [rows of Q]
  int* part;           // [slab][K range][M][128] int32 partial sums
  unsigned* counters;  // [slab] arrivals
  int M, num_kb;
  int n_rows;  // rows of Q
  int n_out;   // output columns
  int ksplit;
};

__device__ __forceinline__ void tc_mma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <bool GLU, bool OUT_F32>
__global__ void __launch_bounds__(kI8DecThreads, 2)
    k_decode_int8(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, DecodeInt8Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* sW = smem;
  uint8_t* sX = sW + kI8DecStages * kI8WStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(sX + kI8DecStages * kI8XStage);
  uint64_t* empty = full + kI8DecStages;
  uint64_t* acc_full = empty + kI8DecStages;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile unsigned* arrival = reinterpret_cast<volatile unsigned*>(tmem_slot + 2);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int ks = p.ksplit;
  const int slab = static_cast<int>(blockIdx.x) / ks, rank = static_cast<int>(blockIdx.x) % ks;
  const int n0 = slab * kI8Rows;
  const int kb0 = static_cast<int>(static_cast<long long>(rank) * p.num_kb / ks);
  const int kb1 = static_cast<int>(static_cast<long long>(rank + 1) * p.num_kb / ks);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kI8DecStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 64);
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
      const int first = min(kb1, kb0 + kI8DecStages);
      for (int kb = kb0; kb < first; ++kb) {  // every stage is free at the start
        const int st = kb - kb0;
        mbar_arrive_expect_tx(&full[st], kI8WStage + kI8XStage);
        tma_load_2d(sW + st * kI8WStage, &tm_w, &full[st], kb * 128, n0);
      }
      grid_dep_wait();  // the row pass is complete: its codes may be read
      for (int kb = kb0; kb < kb1; ++kb) {
        if (kb >= first) {
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], kI8WStage + kI8XStage);
          tma_load_2d(sW + s * kI8WStage, &tm_w, &full[s], kb * 128, n0);
        }
        tma_load_2d(sX + s * kI8XStage, &tm_x, &full[s], kb * 128, 0);
        ++issued;
        if (++s == kI8DecStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      grid_dep_launch();
      if (ok) {
        // no arrival on this CTA's barriers (an MMA commit completes asynchronously) may be in flight at its exit
        for (int i = 0; i < kI8DecStages; ++i) {
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag)) break;
          if (++s == kI8DecStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) {
        const int pending = issued < kI8DecStages ? issued : kI8DecStages;
        for (int i = 1; i <= pending; ++i) {
          int st = s - i;
          uint32_t pp = ph;
          if (st < 0) {
            st += kI8DecStages;
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
      const uint32_t idesc = make_idesc_i8(kI8Rows, kI8Tok);
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full[s], ph, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t a_addr = smem_u32(sW + s * kI8WStage);
        const uint32_t b_addr = smem_u32(sX + s * kI8XStage);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // MMA k of every stage into accumulator k: four independent chains
          tc_mma_i8(tmem_base + static_cast<uint32_t>(k * kI8Tok), make_sdesc_sw128(a_addr + k * 32),
                    make_sdesc_sw128(b_addr + k * 32), idesc, kb != kb0 ? 1u : 0u);
        tc_commit(&empty[s]);
        if (++s == kI8DecStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      tc_commit(ok ? acc_full : drain);
      if (!ok) {
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int t = static_cast<int>(threadIdx.x) - 64;
    const int row = q * 32 + lane;  // row of Q within the slab
    grid_dep_wait();
    bool ok = __all_sync(0xffffffffu, mbar_wait(acc_full, 0, abort_flag));
    int v[kI8Tok];
#pragma unroll
    for (int j = 0; j < kI8Tok; ++j) v[j] = 0;
    if (ok) {
      tc_fence_after_sync();
      const uint32_t lanes = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        uint32_t r[16];
        tmem_ld16(lanes + a * kI8Tok, r);
        tmem_ld_wait();
        reg_fence16(r);
#pragma unroll
        for (int j = 0; j < kI8Tok; ++j) v[j] += static_cast<int>(r[j]);
      }
    }
    bool writer = true;
    if (ks > 1) {
      const size_t rec = static_cast<size_t>(slab) * static_cast<size_t>(ks);
      const size_t plane = static_cast<size_t>(p.M) * kI8Rows;
      int* mine = p.part + (rec + rank) * plane + row;
#pragma unroll
      for (int m = 0; m < kI8Tok; ++m)
        if (m < p.M) __stcg(mine + m * kI8Rows, v[m]);
      named_bar_sync(1, 128);  // the CTA's partials come before its arrival (barrier, then release)
      // Acquire-release at GPU scope: releases this CTA's partials and, for the last arrival, acquires the other
      // ranges'. An arrival that carries kI8Gave marks the slab's sums as incomplete.
      if (t == 0) *arrival = atom_add_acq_rel_gpu(p.counters + slab, *abort_flag ? 1u + kI8Gave : 1u);
      named_bar_sync(1, 128);
      const unsigned before = *arrival;
      writer = (before & (kI8Gave - 1u)) == static_cast<unsigned>(ks - 1);
      if (writer) {
        ok = ok && before < kI8Gave;
        for (int rr = 0; rr < ks; ++rr) {
          if (rr == rank) continue;
          const int* src = p.part + (rec + rr) * plane + row;
#pragma unroll
          for (int m = 0; m < kI8Tok; ++m)
            if (m < p.M) v[m] += __ldcg(src + m * kI8Rows);
        }
      }
    }
    if (writer) {
      const int n = n0 + row;
      // a sum that a failed wait left incomplete is written as NaN (the status word reports the timeout)
      const float sc = !ok || *abort_flag ? __int_as_float(0x7fc00000) : n < p.n_rows ? __ldg(p.scale + n) : 0.f;
      // rows 32b + j (gate) and 32b + 16 + j (up) are lanes j and j + 16 of one warp
      const int col = GLU ? ((n0 + q * 32) >> 1) + (lane & 15) : n;
      const bool mine = col < p.n_out && (!GLU || lane < 16);
#pragma unroll
      for (int m = 0; m < kI8Tok; ++m) {
        if (m >= p.M) break;
        float o = static_cast<float>(v[m]) * __ldcg(p.rho + m) * sc;
        if (GLU) o = int8_swiglu(o, __shfl_down_sync(0xffffffffu, o, 16));
        if (mine) {
          if (OUT_F32)
            static_cast<float*>(p.y)[static_cast<size_t>(m) * p.n_out + col] = o;
          else
            static_cast<uint16_t*>(p.y)[static_cast<size_t>(m) * p.n_out + col] =
                static_cast<uint16_t>(pack_bf16x2(o, 0.f) & 0xFFFFu);
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem_base, 64);
}

}  // namespace fn
