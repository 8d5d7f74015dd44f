// pair_gemm.cuh — the persistent CTA-pair matrix product (tcgen05 cta_group::2) behind the 8-bit integer
// projection and the vocabulary head: C = A . B^T with one epilogue functor per use.
//
// Two CTAs of a cluster share each MMA of M = 256 rows: each stages its own 128 rows of A and half of the tile's
// B rows (TMA into a ring of 128-byte-swizzled stages), the leader issues the MMAs, and each CTA's tensor memory
// holds the accumulator of its own 128 rows (two of them, so that a tile's epilogue runs under the next tile's
// MMAs). Unlike the deferred-norm kernel of fused_gemm_pair.cuh no warps read the staged x tiles: row statistics
// come from a row pass before, which these operators need anyway (8-bit codes, 1/rms of the head). A tile may
// therefore go to any pair, and pairs take tiles round robin in bands of `band` row tiles, row tile fastest: the
// pairs running at one moment cover a compact block of C and share its A and B tiles in L2.
//
// Operands. bf16 (kind::f16, fp32 accumulator) or int8 (kind::i8, exact int32 accumulator); a stage holds 128
// bytes of K per row (64 bf16, 128 int8). A bf16 operand may also be "MN-major": stored [K][rows], as a
// transposed factor of a gradient is; its stage is two boxes of 64 k x 64 rows, each 64 lines of 128 bytes, brought by one
// copy where the rows are whole blocks of 64 (dx and dW* at 2048 x 4096 x 16000: 340 us, 370 with a copy per box). Tiles of an
// MN-major B are multiples of 128 wide, so that every box starts on a 128-byte line: boxes that start in the middle of one
// took 1.8 times as long (517 x 576 outputs, k = 50257: 125 against 69 us with narrower, aligned tiles). The last column
// tile is only as wide as its columns need.
//
// Two products that share nothing but the grid may run as one launch (jobs 0 and 1): a pair takes its items of job 0,
// usually few and long, and then its share of job 1's many short ones, which evens out what job 0 left uneven.
//
// Accumulation. The tensor core adds into its fp32 accumulator without rounding to nearest, so a long sum drifts (at
// k = 4096 a logit's relative error is near 4e-6). An epilogue that needs better takes the sum in chunks of `kchunk` stages,
// which it adds in its own registers.
//
// Warps: 0 = TMA producer, 1 = MMA issuer (leader) and tensor memory, the others epilogue, Epi::kParts (2 or 4) per lane
// quarter. Four leave each thread 96 registers instead of 168. The loss has four; two take 1 to 8 % less at the rows it serves
// (2048 x 576 x 49152: 82 against 86 to 89 us, 2048 x 4096 x 32000: 345 against 350, 64 x 4096 x 32000: 56.6 against 57.8).
// The others have two: P's epilogue spills with four (170 us against 165 at 2048 x 4096 x 16000).
//
// What bounds it: the tensor pipe, 86 % of cycles busy at 2048 x 4096 x 16000 (the clock then falls to 1.55 GHz: 1.6 PFLOP/s
// for one launch, 1.3 back to back under the power cap); the L2 at k of a few stages or narrow tiles. One warp issues loads
// and one MMAs, whole warps whose lane 0 issues, because both have little time: addresses and descriptors are offsets from
// bases taken once per item, and placing the items in one thread, with its divisions, had cost 13 % (8-bit 2048 x 4096 x
// 22016: 133 against 117 us).
#pragma once

#include <type_traits>

#include "sm100.cuh"

namespace fn {

constexpr int kPgStages = 6;
constexpr int kPgTileBytes = 16 * 1024;  // A or B of one stage: 128 rows x 128 bytes
constexpr int kPgOutBytes = 32 * 64;     // per epilogue warp: 32 rows x 64 bytes on their way out

__host__ __device__ constexpr int pair_gemm_threads(int parts) { return 64 + 128 * parts; }
__host__ __device__ constexpr int pair_gemm_smem_bytes(int parts) {
  return 1024 + kPgStages * 2 * kPgTileBytes + 4 * parts * kPgOutBytes + 1024;
}

struct PairGemmParams {
  int M, N;         // rows and columns of C
  int num_kb;       // stages along K
  int kchunk;       // stages per accumulation (an epilogue that takes only whole sums: num_kb)
  int bn;           // tile width: a multiple of 32 (MN-major B: of 128), at most 256
  int num_m_tiles;  // of 256 rows
  int num_n_tiles;
  int band;         // row tiles per band
  int ksplit;       // K ranges; range z of a tile goes to the epilogue as plane z
  int early;        // PgEarly: operands that do not depend on the previous kernel of the stream
  int live_is_k;    // what *live counts: rows of C, or (1) k
  const int* live;  // null, or a count on the device that replaces M (at most M) or num_kb (at most so many stages)
  int b_blocks;     // MN-major B: its map has blocks of 64 columns as a third dimension, one copy per stage
  int extra;        // job 1: items that a pair with one item less of job 0 takes first, in exchange
  unsigned* failed;  // null, or a word that is set to 1 if tiles are left unfinished because a wait ran out
};

// Operands that may be fetched before the previous kernel has completed. That kernel must itself have waited for all
// work before it (griddepcontrol.wait) before it let this one start, so that what is fetched early is in place.
enum PgEarly { PG_EARLY_NONE = 0, PG_EARLY_B = 1, PG_EARLY_AB = 2 };

enum PgKind { PG_BF16 = 0, PG_I8 = 1 };

// kind::i8 on a CTA pair, int32 accumulate.
__device__ __forceinline__ void tc_mma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor for kind::i8: signed 8-bit A and B, K-major, int32 D, shape M x N.
__host__ __device__ constexpr uint32_t make_idesc_i8(int m, int n) {
  return (2u << 4)                                // D format: s32
         | (1u << 7)                              // A format: s8
         | (1u << 10)                             // B format: s8
         | (static_cast<uint32_t>(n >> 3) << 17)  // N / 8
         | (static_cast<uint32_t>(m >> 4) << 24);  // M / 16
}

// Matrix descriptor of an MN-major operand: 64-wide blocks of 64 k lines (128 bytes each, 128-byte swizzle over
// groups of 8 lines); the next block of 64 rows is 8 KB on (leading byte offset), the next 8 k 1 KB on (stride
// byte offset).
__device__ __forceinline__ uint64_t make_sdesc_mn_sw128(uint32_t smem_addr) {
  return static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(8192 >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// What an epilogue warp works on: 32 rows of one tile (row0 + lane is this thread's) and columns col0 .. of it.
struct PgTile {
  uint32_t t_row;  // tensor-memory address of this warp's lanes, accumulator column 0
  int row0;        // first row of the warp's lane quarter
  int n0, width;   // the tile's columns
  int part;        // chunks part, part + kParts, ... of the tile are this warp's (the quarter's warps trade from tile to tile)
  int nt, kz;      // column tile and K range
  int M;           // rows of C
  bool empty;      // no k at all: the accumulator holds nothing and counts as zero
  int chunk, chunks;  // accumulations of this tile: which one run() has before it, and how many
  uint8_t* stage;  // this warp's staging buffer
};

// Copy a staged block of 32 rows x 64 bytes out, 8 rows x 64 bytes per warp store. `y` is the tensor, `ldb` its
// row stride in bytes, `colb` the block's first column in bytes, `endb` the row's length in bytes (a multiple of
// 16). The block was staged by pg_put: 16-byte piece j of row r at r * 64 + ((j ^ (r >> 1)) & 3) * 16.
__device__ __forceinline__ void pg_put(uint8_t* stage, int lane, int j, uint4 v) {
  *reinterpret_cast<uint4*>(stage + lane * 64 + (((j ^ (lane >> 1)) & 3) << 4)) = v;
}
__device__ __forceinline__ void pg_flush(uint8_t* stage, int lane, void* y, size_t ldb, int row0, int M, long long colb,
                                         long long endb) {
  __syncwarp();
  const int seg = lane & 3;
  const long long at = colb + seg * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rr = 8 * i + (lane >> 2);
    const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 64 + (((seg ^ (rr >> 1)) & 3) << 4));
    if (row0 + rr < M && at < endb)
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(y) + static_cast<size_t>(row0 + rr) * ldb + at) = v;
  }
  __syncwarp();  // the staging buffer is read before the next block overwrites it
}

// One product: operand layouts and epilogue.
template <bool A_MN_, bool B_MN_, class Epi_>
struct PgJob {
  static constexpr bool A_MN = A_MN_, B_MN = B_MN_;
  using Epi = Epi_;
  using Params = typename Epi_::Params;
};

// The empty second job.
struct PgNoEpi {
  static constexpr int kParts = 2;
  struct Params {};
  __device__ __forceinline__ PgNoEpi(const Params&, const PairGemmParams&, const PgTile&, int) {}
  __device__ __forceinline__ void run(const Params&, const PairGemmParams&, const PgTile&, int) {}
};
using PgNoJob = PgJob<false, false, PgNoEpi>;

// What the device knows of one job: sizes after *live has been read, and where item t lies.
struct PgPlan {
  int rows, num_kb, m_tiles, tiles, items;
  __device__ __forceinline__ PgPlan(const PairGemmParams& p, int k_per_stage) {
    rows = p.M, num_kb = p.num_kb;
    if (p.live != nullptr) {
      const int live = __ldcg(p.live);
      if (p.live_is_k)
        num_kb = (live + k_per_stage - 1) / k_per_stage;
      else
        rows = live;
    }
    m_tiles = (rows + 255) >> 8;
    tiles = m_tiles * p.num_n_tiles;
    items = tiles * p.ksplit;
  }
};

struct PgItem {
  int job, mt, nt, kz, kb0, kb1, width, wide;  // job -1: no more; width: columns; wide: the MMA's N
};

// A warp's walk through its pair's items. Placing one takes a few integer divisions, over 500 cycles in one thread and
// more than a short tile's MMAs leave between two tiles, so the lanes place the next 32 items at once.
template <class Place>
struct PgWalk {
  const Place& place;  // place(i, item): item i of the pair
  PgItem mine;
  int lane, i = 0;
  __device__ __forceinline__ PgWalk(const Place& p, int l) : place(p), lane(l) {}
  __device__ __forceinline__ bool next(PgItem& it) {
    if ((i & 31) == 0) place(i + lane, mine);
    const int src = i++ & 31;
    it.job = __shfl_sync(0xffffffffu, mine.job, src);
    it.mt = __shfl_sync(0xffffffffu, mine.mt, src);
    it.nt = __shfl_sync(0xffffffffu, mine.nt, src);
    it.kz = __shfl_sync(0xffffffffu, mine.kz, src);
    it.kb0 = __shfl_sync(0xffffffffu, mine.kb0, src);
    it.kb1 = __shfl_sync(0xffffffffu, mine.kb1, src);
    it.width = __shfl_sync(0xffffffffu, mine.width, src);
    it.wide = __shfl_sync(0xffffffffu, mine.wide, src);
    return it.job >= 0;
  }
};

template <int KIND, class J0, class J1, bool TWO>
__device__ __forceinline__ void pair_gemm_body(const CUtensorMap& tm_a0, const CUtensorMap& tm_b0, const PairGemmParams& p0,
                                               const typename J0::Params& ep0, const CUtensorMap& tm_a1,
                                               const CUtensorMap& tm_b1, const PairGemmParams& p1,
                                               const typename J1::Params& ep1) {
  static_assert(KIND == PG_BF16 || (!J0::A_MN && !J0::B_MN && !TWO), "8-bit operands are K-major");
  constexpr int kElem = KIND == PG_I8 ? 1 : 2;
  constexpr int kK = 128 / kElem;  // k per stage
  constexpr int kParts = J0::Epi::kParts;
  static_assert(!TWO || J0::Epi::kParts == J1::Epi::kParts, "one set of epilogue warps");

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* sA = smem;
  uint8_t* sB = sA + kPgStages * kPgTileBytes;
  uint8_t* sOut = sB + kPgStages * kPgTileBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sOut + 4 * kParts * kPgOutBytes);  // used in the leader
  uint64_t* empty = full + kPgStages;
  uint64_t* acc_full = empty + kPgStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2], used in the leader
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPgStages; ++s) {
      mbar_init(&full[s], 1);   // the leader's expect-tx arrival covers both CTAs' bytes
      mbar_init(&empty[s], 1);  // the MMA's commit (multicast to both CTAs)
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8 * kParts);  // the epilogue warps of both CTAs
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a0);
    tma_prefetch_desc(&tm_b0);
    if (TWO) {
      tma_prefetch_desc(&tm_a1);
      tma_prefetch_desc(&tm_b1);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before either touches the other's
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  // The previous kernel's outputs (our inputs, or buffers we overwrite) are complete. Early operands do not wait for that;
  // their producer does once it needs the others, the epilogue always does. Early operands exclude *live and a second job.
  if (p0.early == PG_EARLY_NONE || warp >= 2) grid_dep_wait();

  const int cl = static_cast<int>(blockIdx.x) >> 1, ncl = static_cast<int>(gridDim.x) >> 1;
  const PgPlan plan0(p0, kK);
  const PgPlan plan1 = TWO ? PgPlan(p1, kK) : plan0;
  // Items t of a job: bands of `band` row tiles, row tile fastest, K ranges outermost.
  auto place = [&](const PairGemmParams& p, const PgPlan& pl, bool b_mn, int t, PgItem& it) {
    it.kz = t / pl.tiles;
    const int u = t - it.kz * pl.tiles;
    const int per_band = p.band * p.num_n_tiles;
    const int b = u / per_band, r = u - b * per_band;
    const int in_band = min(p.band, pl.m_tiles - b * p.band);
    it.mt = b * p.band + r % in_band;
    it.nt = r / in_band;
    it.kb0 = static_cast<int>(static_cast<long long>(it.kz) * pl.num_kb / p.ksplit);
    it.kb1 = static_cast<int>(static_cast<long long>(it.kz + 1) * pl.num_kb / p.ksplit);
    it.width = min(p.bn, p.N - it.nt * p.bn);
    it.wide = b_mn ? (it.width + 127) & ~127 : (it.width + 31) & ~31;
  };
  // Item i of this pair. Job 0 goes round robin. Of job 1, the pairs that got one item less of job 0 first take `extra`
  // items each, the rest goes round robin.
  const int n0 = (plan0.items - cl + ncl - 1) / ncl;  // 0 or less: none
  const int heavy = plan0.items % ncl;
  const int lights = heavy ? ncl - heavy : 0;
  const int light_extra = TWO && lights ? min(p1.extra, plan1.items / lights) : 0;
  auto item_at = [&](int i, PgItem& it) {
    it = {-1, 0, 0, 0, 0, 0, 0, 0};
    if (!TWO || i < n0) {
      const long long t = cl + static_cast<long long>(i) * ncl;  // the lanes look past the last item
      if (t >= plan0.items) return;
      it.job = 0;
      place(p0, plan0, J0::B_MN, static_cast<int>(t), it);
      return;
    }
    const int j = i - n0;
    long long t;
    if (heavy && cl >= heavy) {
      t = j < light_extra ? (cl - heavy) + static_cast<long long>(j) * lights
                          : lights * light_extra + cl + static_cast<long long>(j - light_extra) * ncl;
    } else {
      t = lights * light_extra + cl + static_cast<long long>(j) * ncl;
    }
    if (t >= plan1.items) return;
    it.job = 1;
    place(p1, plan1, J1::B_MN, static_cast<int>(t), it);
  };
  PgWalk<decltype(item_at)> walk(item_at, lane);
  PgItem it;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer (both CTAs; lane 0 issues)
    {
      int s = 0, issued = 0;
      uint32_t ph = 0;
      bool ok = true;
      auto bytes_of = [&](const PgItem& it, const PairGemmParams& p, bool b_mn) {
        return static_cast<uint32_t>(kPgTileBytes + (b_mn && !p.b_blocks ? it.wide * 64 : p.bn * 64));
      };
      // One thread issues everything for a stage within the time of its MMAs (512 cycles at most), so addresses are kept
      // as offsets from a few bases.
      const uint32_t full0 = dsmem_addr(&full[0], 0), a0 = smem_u32(sA), b0 = smem_u32(sB);
      auto load_a = [&](bool mn, const CUtensorMap* tm, int st, int k, int m0) {
        const uint32_t bar = full0 + 8u * st, dst = a0 + static_cast<uint32_t>(st * kPgTileBytes);
        if (mn) {
          tma_load_3d_pair_at(dst, tm, bar, 0, k, m0 >> 6);
        } else {
          tma_load_2d_pair_at(dst, tm, bar, k, m0);
        }
      };
      // K-major: one box of bn / 2 rows, of which a narrower last tile uses the first ones
      auto load_b = [&](bool mn, bool blocks, const CUtensorMap* tm, int st, int k, int n0, int wide) {
        const uint32_t bar = full0 + 8u * st, dst = b0 + static_cast<uint32_t>(st * kPgTileBytes);
        if (mn && blocks) {
          tma_load_3d_pair_at(dst, tm, bar, 0, k, n0 >> 6);
        } else if (mn) {
          tma_load_2d_pair_at(dst, tm, bar, n0, k);
          if (wide > 128) tma_load_2d_pair_at(dst + 8192, tm, bar, n0 + 64, k);
        } else {
          tma_load_2d_pair_at(dst, tm, bar, k, n0);
        }
      };
      int ahead = 0;  // stages whose B is already on its way
      bool more = walk.next(it);
      if (!TWO && p0.early == PG_EARLY_B) {
        if (more) {
          ahead = min(kPgStages, it.kb1 - it.kb0);
          if (lane == 0)
            for (int st = 0; st < ahead; ++st) {  // every stage is free at the start
              if (leader) mbar_arrive_expect_tx(&full[st], 2 * bytes_of(it, p0, J0::B_MN));
              load_b(J0::B_MN, p0.b_blocks, &tm_b0, st, (it.kb0 + st) * kK, it.nt * p0.bn + static_cast<int>(rank) * (it.wide / 2), it.wide);
            }
        }
        grid_dep_wait();
      }
      for (; ok && more; more = walk.next(it)) {
        const bool second = TWO && it.job == 1;
        const PairGemmParams& p = second ? p1 : p0;
        const CUtensorMap* tm_a = second ? &tm_a1 : &tm_a0;
        const CUtensorMap* tm_b = second ? &tm_b1 : &tm_b0;
        const bool a_mn = second ? J1::A_MN : J0::A_MN, b_mn = second ? J1::B_MN : J0::B_MN;
        const uint32_t stage_bytes = 2 * bytes_of(it, p, b_mn);
        const int m0 = it.mt * 256 + static_cast<int>(rank) * 128;
        const int n0 = it.nt * p.bn + static_cast<int>(rank) * (it.wide / 2);
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          if (issued >= ahead && !__all_sync(0xffffffffu, mbar_wait_cluster(&empty[s], ph ^ 1u, abort_flag))) {
            ok = false;
            break;
          }
          if (lane == 0) {
            if (issued >= ahead) {
              if (leader) mbar_arrive_expect_tx(&full[s], stage_bytes);
              load_b(b_mn, p.b_blocks, tm_b, s, kb * kK, n0, it.wide);
            }
            load_a(a_mn, tm_a, s, kb * kK, m0);
          }
          __syncwarp();
          ++issued;
          if (++s == kPgStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      grid_dep_launch();  // all loads issued: the next kernel may be scheduled onto SMs as they free up
      if (ok && lane == 0) {
        // The release of the last use of every stage, so that no arrival on this CTA's barriers (an MMA commit
        // completes asynchronously) is still in flight when the CTA exits.
        for (int i = 0; i < kPgStages; ++i) {
          if (!mbar_wait_cluster(&empty[s], ph ^ 1u, abort_flag)) break;
          if (++s == kPgStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok && leader && lane == 0) {
        // Gave up: let the pair's copies still in flight land (bounded) before shared memory goes.
        const int pending = issued < kPgStages ? issued : kPgStages;
        for (int i = 1; i <= pending; ++i) {
          int st = s - i;
          uint32_t pp = ph;
          if (st < 0) {
            st += kPgStages;
            pp ^= 1u;
          }
          const unsigned long long t0 = globaltimer_ns();
          while (!mbar_try_wait_cluster(&full[st], pp) && globaltimer_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ pair MMA issuer (leader)
    if (leader) {  // lane 0 issues
      int s = 0;
      uint32_t ph = 0;
      int acc = 0;
      uint32_t acc_ph = 0;
      bool ok = true;
      while (ok && walk.next(it)) {
        const bool second = TWO && it.job == 1;
        const int kchunk = second ? p1.kchunk : p0.kchunk;
        const bool a_mn = second ? J1::A_MN : J0::A_MN, b_mn = second ? J1::B_MN : J0::B_MN;
        const uint32_t idesc = KIND == PG_I8 ? make_idesc_i8(256, it.wide)
                                             : make_idesc_bf16(256, it.wide) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
        // Descriptors of stage 0; a stage on adds 16 KB, an MMA on 32 bytes of every row (K-major) or 16 lines (MN-major),
        // all in units of 16 bytes.
        const uint32_t a_addr = smem_u32(sA), b_addr = smem_u32(sB);
        const uint64_t da0 = a_mn ? make_sdesc_mn_sw128(a_addr) : make_sdesc_sw128(a_addr);
        const uint64_t db0 = b_mn ? make_sdesc_mn_sw128(b_addr) : make_sdesc_sw128(b_addr);
        const uint64_t a_step = a_mn ? 128 : 2, b_step = b_mn ? 128 : 2;
        int kb = it.kb0;
        do {  // one accumulation; a tile without k still hands its (empty) accumulator on
          const int end = min(kb + kchunk, it.kb1);
          if (!__all_sync(0xffffffffu, mbar_wait_cluster(&acc_empty[acc], acc_ph ^ 1u, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 256);
          for (int first = kb; kb < end; ++kb) {
            if (!__all_sync(0xffffffffu, mbar_wait_cluster(&full[s], ph, abort_flag))) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            uint64_t da = da0 + static_cast<uint64_t>(s * (kPgTileBytes / 16));
            uint64_t db = db0 + static_cast<uint64_t>(s * (kPgTileBytes / 16));
#pragma unroll
            for (int k = 0; k < 4; ++k, da += a_step, db += b_step) {
              const uint32_t accumulate = (kb != first || k != 0) ? 1u : 0u;
              if (lane != 0) continue;
              if (KIND == PG_I8)
                tc_mma_i8_pair(d_tmem, da, db, idesc, accumulate);
              else
                tc_mma_bf16_pair(d_tmem, da, db, idesc, accumulate);
            }
            if (lane == 0) tc_commit_pair_mc(&empty[s], 0x3);  // frees stage s in both CTAs once read
            __syncwarp();
            if (++s == kPgStages) {
              s = 0;
              ph ^= 1u;
            }
          }
          if (!ok) break;
          if (lane == 0) tc_commit_pair_mc(&acc_full[acc], 0x3);
          __syncwarp();
          acc ^= 1;
          if (acc == 0) acc_ph ^= 1u;
        } while (kb < it.kb1);
      }
      if (!ok && lane == 0) {
        tc_commit_pair_mc(drain, 0x1);
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;
    const uint32_t leader_acc_empty0 = dsmem_addr(&acc_empty[0], 0);
    const uint32_t leader_acc_empty1 = dsmem_addr(&acc_empty[1], 0);
    int acc = 0;
    uint32_t acc_ph = 0;
    // One tile: false, for the whole warp, once a wait gave up.
    auto finish = [&](auto* job, const PairGemmParams& p, const auto& ep, const PgPlan& pl, int turn) {
      using Epi = typename std::remove_pointer_t<decltype(job)>::Epi;
      PgTile tile;
      tile.row0 = it.mt * 256 + static_cast<int>(rank) * 128 + q * 32;
      tile.n0 = it.nt * p.bn;
      tile.width = it.width;
      tile.part = (((warp - 2) >> 2) + turn) % kParts;
      tile.nt = it.nt;
      tile.kz = it.kz;
      tile.M = pl.rows;
      tile.empty = it.kb0 == it.kb1;
      tile.chunks = max(1, (it.kb1 - it.kb0 + p.kchunk - 1) / p.kchunk);
      tile.stage = sOut + (warp - 2) * kPgOutBytes;
      Epi epi(ep, p, tile, lane);  // row parameters are on their way while the MMAs finish
      for (tile.chunk = 0; tile.chunk < tile.chunks; ++tile.chunk) {
        tile.t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * 256);
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(&acc_full[acc], acc_ph, abort_flag))) return false;
        tc_fence_after_sync();
        epi.run(ep, p, tile, lane);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (leader)
            mbar_arrive(&acc_empty[acc]);
          else
            mbar_arrive_remote(acc == 0 ? leader_acc_empty0 : leader_acc_empty1);
        }
        acc ^= 1;
        if (acc == 0) acc_ph ^= 1u;
      }
      return true;
    };
    bool ok = true;
    for (int turn = 0; ok && walk.next(it); ++turn) {
      if (TWO && it.job == 1)
        ok = finish(static_cast<J1*>(nullptr), p1, ep1, plan1, turn);
      else
        ok = finish(static_cast<J0*>(nullptr), p0, ep0, plan0, turn);
    }
    if (!ok && lane == 0 && p0.failed != nullptr) atomicExch(p0.failed, 1u);
  }

  // ------------------------------------------------------------------ teardown
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while the other may still signal its barriers
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

template <int KIND, class J>
__global__ void __launch_bounds__(pair_gemm_threads(J::Epi::kParts), 1)
    k_pair_gemm(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                const __grid_constant__ PairGemmParams p, const __grid_constant__ typename J::Params ep) {
  const PgNoEpi::Params none;
  pair_gemm_body<KIND, J, PgNoJob, false>(tm_a, tm_b, p, ep, tm_a, tm_b, p, none);
}

// Two bf16 products in one launch.
template <class J0, class J1>
__global__ void __launch_bounds__(pair_gemm_threads(J0::Epi::kParts), 1)
    k_pair_gemm2(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_b0,
                 const __grid_constant__ PairGemmParams p0, const __grid_constant__ typename J0::Params ep0,
                 const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_b1,
                 const __grid_constant__ PairGemmParams p1, const __grid_constant__ typename J1::Params ep1) {
  pair_gemm_body<PG_BF16, J0, J1, true>(tm_a0, tm_b0, p0, ep0, tm_a1, tm_b1, p1, ep1);
}

}  // namespace fn
