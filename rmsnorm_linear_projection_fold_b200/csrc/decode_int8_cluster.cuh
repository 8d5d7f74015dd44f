// decode_int8_cluster.cuh — the 8-bit integer projection for at most 16 rows in one launch: the rows are quantized by the
// CTAs that multiply them.
//
// As in decode_int8.cuh, rows of Q form the MMA's M side and the tokens its N side, and the contraction of a slab of rows is
// cut into K ranges. A slab has 128 rows, or 96, 64 or 32 (the MMA's other rows are not used) where that fills more of the
// SMs' two places each; here the ranges of a slab are the CTAs of a cluster. Each reads only its own K range of x,
// takes the partial maximum and sum of squares of every row, exchanges them with its cluster (distributed shared memory),
// and writes the codes of its range straight into the MMA's operand layout. Partial sums go to the rank that finishes
// their token, again through distributed shared memory: no workspace and no second launch. Each slab's cluster reads all of
// x from L2, at most a quarter of its Q bytes.
//
// Measured (warm): 1 x 576 -> 960 6.8 us (row pass and separate product: 4.5 + 7.8), all latency: launch, x, the exchange, the
// MMAs' commit, the second exchange. 4 x 4096 -> 12288 15 us, of which Q's 50 MB need 7.8: the ring holds a third of Q while
// the codes are made, the rest streams after.
//
// Warps: 0 = TMA producer, 1 = tensor memory + MMA issuer, 2..9 = quantization, then epilogue (two per lane quarter).
#pragma once

#include "decode_int8.cuh"

namespace fn {

constexpr int kI8cThreads = 320;
constexpr int kI8cMaxRanks = 8;
constexpr int kI8cRedSlots = 16;  // ranks (a power of two) x tokens per rank

struct Int8ClusterParams {
  const uint16_t* x;   // [M][K]
  void* y;
  const float* scale;  // [rows of Q]
  int M, K, num_kb;
  int n_rows;  // rows of Q
  int n_out;   // output columns
  int ranks;   // CTAs per slab
  int rows;    // of a slab: a multiple of 32, at most 128
  int stages;  // of the ring
  int max_kb;  // of a rank
  float eps;
  int norm;
};

// Per K block: 8 rows of codes for at most 8 tokens, else 16.
__host__ __device__ constexpr int int8_cluster_code_bytes(int M) { return M <= 8 ? 1024 : 2048; }
// The MMA reads 128 rows whatever the slab has: the codes (16 KB at most past the last stage's start) or what follows them.
__host__ __device__ constexpr int int8_cluster_smem_bytes(int M, int max_kb, int stages, int rows) {
  return 1024 + stages * rows * 128 + (kI8Rows - rows) * 128 + max_kb * int8_cluster_code_bytes(M) + kI8cRedSlots * 512 + 2560;
}

// Load 8 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

__device__ __forceinline__ void dsmem_st_b32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void dsmem_st_b64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

template <bool GLU, bool OUT_F32>
__global__ void __launch_bounds__(kI8cThreads, 2)
    k_decode_int8_cluster(const __grid_constant__ CUtensorMap tm_w, Int8ClusterParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const int code_bytes = int8_cluster_code_bytes(p.M);
  uint8_t* sW = smem;
  const int stage_bytes = p.rows * 128;
  uint8_t* sX = sW + p.stages * stage_bytes;
  int* red = reinterpret_cast<int*>(sX + p.max_kb * code_bytes);            // [rank][token of mine][128]
  uint2* stat = reinterpret_cast<uint2*>(red + kI8cRedSlots * 128);         // [rank][16]: magnitude bits, sum of squares
  float* rho = reinterpret_cast<float*>(stat + kI8cMaxRanks * 16);          // [16]
  uint32_t* failed = reinterpret_cast<uint32_t*>(rho + 16);                 // [rank][8]: by each of its epilogue warps
  uint64_t* full = reinterpret_cast<uint64_t*>(failed + kI8cMaxRanks * 8);  // [16 at most]
  uint64_t* empty = full + 16;
  uint64_t* acc_full = empty + 16;
  uint64_t* codes_ready = acc_full + 1;
  uint64_t* drain = codes_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int ranks = p.ranks;
  const int slab = static_cast<int>(blockIdx.x) / ranks, rank = static_cast<int>(blockIdx.x) % ranks;
  const int n0 = slab * p.rows;
  const int kb0 = rank * p.num_kb / ranks, kb1 = (rank + 1) * p.num_kb / ranks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(codes_ready, 8);
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_init_fence();
    // a hint only: Q may still be written by the kernel before this one
    for (int kb = kb0; kb < min(kb1, kb0 + p.stages); ++kb) tma_prefetch_l2_2d(&tm_w, kb * 128, n0);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 64);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  cluster_arrive();  // with the wait below: no CTA writes into one that has not started
  grid_dep_wait();

  if (warp == 0) {
    int s = 0, kb = kb0;
    uint32_t ph = 0;
    bool ok = true;
    const int first = min(kb1, kb0 + p.stages);
    auto load = [&]() {
      mbar_arrive_expect_tx(&full[s], stage_bytes);
      tma_load_2d(sW + s * stage_bytes, &tm_w, &full[s], kb * 128, n0);
    };
    auto advance = [&]() {
      if (++s == p.stages) {
        s = 0;
        ph ^= 1u;
      }
    };
    if (lane == 0) {
      for (; kb < first; ++kb) {
        load();
        advance();
      }
    }
    __syncwarp();
    cluster_wait();
    cluster_sync_all();  // the rows' statistics have been exchanged
    if (lane == 0) {
      for (; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        load();
        advance();
      }
      grid_dep_launch();
      if (ok) {
        // no arrival on this CTA's barriers (an MMA commit completes asynchronously) may be in flight at its exit
        for (int i = 0; i < p.stages; ++i) {
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag)) break;
          advance();
        }
      } else {
        const int issued = kb - kb0, pending = issued < p.stages ? issued : p.stages;
        for (int i = 1; i <= pending; ++i) {
          int st = s - i;
          uint32_t pp = ph;
          if (st < 0) {
            st += p.stages;
            pp ^= 1u;
          }
          const unsigned long long t0 = globaltimer_ns();
          while (!mbar_try_wait(&full[st], pp) && globaltimer_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    cluster_wait();
    cluster_sync_all();
    if (lane == 0) {
      const uint32_t idesc = make_idesc_i8(kI8Rows, kI8Tok);
      int s = 0;
      uint32_t ph = 0;
      bool ok = mbar_wait(codes_ready, 0, abort_flag);
      const uint32_t a0 = smem_u32(sW), b0 = smem_u32(sX);
      // at most 8 tokens: what the second group of 8 rows reads (the next block's codes) only reaches unused columns
      for (int kb = kb0; ok && kb < kb1; ++kb) {
        if (!mbar_wait(&full[s], ph, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint64_t da = make_sdesc_sw128(a0 + s * stage_bytes);
        const uint64_t db = make_sdesc_sw128(b0 + (kb - kb0) * code_bytes);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // MMA k of every stage into accumulator k: four independent chains
          tc_mma_i8(tmem_base + static_cast<uint32_t>(k * kI8Tok), da + 2 * k, db + 2 * k, idesc, kb != kb0 ? 1u : 0u);
        tc_commit(&empty[s]);
        if (++s == p.stages) {
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
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ quantization: rows w and w + 8
    const int w = warp - 2;
    constexpr int kHeld = 5;  // 16-byte pieces of a row per lane kept in registers: 1280 k
    const int k0 = kb0 * 128, pieces = (min(kb1 * 128, p.K) - k0) >> 3;  // may be 0: K need not fill its last block
    uint4 held[2][kHeld];
    const uint4* src[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = w + 8 * h;
      src[h] = reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(row < p.M ? row : 0) * p.K + k0);
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        held[h][i] = row < p.M && lane + 32 * i < pieces ? __ldcg(src[h] + lane + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
    }
    cluster_wait();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (w + 8 * h >= p.M) continue;
      uint64_t s2 = 0;
      uint32_t amax = 0;
      auto take = [&](const uint4& v) { int8_take(v, s2, amax); };
#pragma unroll
      for (int i = 0; i < kHeld; ++i) take(held[h][i]);
      for (int c = lane + 32 * kHeld; c < pieces; c += 32) take(__ldcg(src[h] + c));
      uint32_t am = max(amax & 0xFFFFu, amax >> 16);
      am = __reduce_max_sync(0xffffffffu, am);
      const float2 halves = unpack_f32x2(s2);
      const float ss = warp_sum(halves.x + halves.y);
      if (lane < ranks)
        dsmem_st_b64(dsmem_addr(stat + rank * 16 + w + 8 * h, static_cast<uint32_t>(lane)), am, __float_as_uint(ss));
    }
    cluster_sync_all();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = w + 8 * h;
      if (row >= p.M) continue;
      uint32_t am = 0;
      float ss = 0.f;
      for (int r = 0; r < ranks; ++r) {  // the same order in every CTA
        const uint2 v = stat[r * 16 + row];
        am = max(am, v.x);
        ss += __uint_as_float(v.y);
      }
      const Int8Row q(am, ss, p.K, p.eps, p.norm);
      if (lane == 0) rho[row] = q.rho;
      // piece c: codes 8c .. 8c+7 of the range; 128-byte rows, 16-byte columns swizzled by the row
      uint8_t* base = sX + (row >> 3) * 1024 + (row & 7) * 128;
      auto put = [&](int c, const uint4& v) {
        const uint2 o = q.codes(v);
        const int kb = c >> 4, col = (c >> 1) & 7;
        *reinterpret_cast<uint2*>(base + kb * code_bytes + ((col ^ (row & 7)) << 4) + 8 * (c & 1)) = o;
      };
      const int all = (kb1 - kb0) * 16;  // past K the codes are zero (Q's are, too: keeps uninitialised memory out)
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (lane + 32 * i < all) put(lane + 32 * i, held[h][i]);
      for (int c = lane + 32 * kHeld; c < all; c += 32)
        put(c, c < pieces ? __ldcg(src[h] + c) : make_uint4(0u, 0u, 0u, 0u));
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(codes_ready);

    // ------------------------------------------------------------------ partial sums to the ranks that finish them
    const int q = warp & 3, half = w >> 2;
    const int row = q * 32 + lane;  // of the slab
    const bool ok = __all_sync(0xffffffffu, mbar_wait(acc_full, 0, abort_flag));
    int v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0;
    if (ok && 8 * half < p.M) {
      tc_fence_after_sync();
      const uint32_t lanes = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + 8 * half;
      uint32_t r[4][8];
#pragma unroll
      for (int a = 0; a < 4; ++a) tmem_ld8(lanes + a * kI8Tok, r[a]);
      tmem_ld_wait();
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          asm volatile("" : "+r"(r[a][j]));
          v[j] += static_cast<int>(r[a][j]);
        }
    }
    // token m is finished by rank m % ranks, as its token m / ranks
    const int per = (kI8Tok + ranks - 1) / ranks;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int m = 8 * half + j;
      if (m >= p.M) break;
      dsmem_st_b32(dsmem_addr(red + (rank * per + m / ranks) * kI8Rows + row, static_cast<uint32_t>(m % ranks)),
                   static_cast<uint32_t>(v[j]));
    }
    if (lane < ranks) dsmem_st_b32(dsmem_addr(failed + rank * 8 + w, static_cast<uint32_t>(lane)), *abort_flag != 0 || !ok ? 1u : 0u);
  }
  tc_fence_before_sync();
  cluster_sync_all();  // partial sums are in place, and no CTA is written to any more
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem_base, 64);
  if (warp >= 2) {
    const int w = warp - 2, q = warp & 3, half = w >> 2;
    const int row = q * 32 + lane, n = n0 + row;
    const bool bad = __any_sync(0xffffffffu, (lane < 8 * ranks && failed[lane] != 0) || (lane + 32 < 8 * ranks && failed[lane + 32] != 0));
    // a sum that a failed wait left incomplete is written as NaN (the status word reports the timeout)
    const float sc = bad ? __int_as_float(0x7fc00000) : row < p.rows && n < p.n_rows ? __ldcg(p.scale + n) : 0.f;
    // rows 32b + j (gate) and 32b + 16 + j (up) are lanes j and j + 16 of one warp
    const int col = GLU ? ((n0 + q * 32) >> 1) + (lane & 15) : n;
    const bool mine = row < p.rows && col < p.n_out && (!GLU || lane < 16);
    const int per = (kI8Tok + ranks - 1) / ranks;
    for (int i = half; i * ranks + rank < p.M; i += 2) {
      const int m = i * ranks + rank;
      int sum = 0;
      for (int r = 0; r < ranks; ++r) sum += red[(r * per + i) * kI8Rows + row];
      float o = static_cast<float>(sum) * rho[m] * sc;
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

}  // namespace fn
