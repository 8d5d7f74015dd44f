// cross_entropy.cuh — softmax cross entropy of the vocabulary head behind the final RMSNorm, and its gradient, without
// keeping the logits.
//
// The head is one more projection behind a norm, so the gain is folded into it and 1/rms deferred ("FlashNorm: Fast
// Normalization for Transformers", Abstract): with r[m] = 1/sqrt(mean(x[m]^2) + eps),
//     l[m, n] = r[m] sum_k x[m, k] W*[n, k],   lse[m] = log sum_n exp(l[m, n]),   loss[m] = lse[m] - l[m, t[m]].
// Forward (more than 32 rows; fewer: cross_entropy_small.cuh): the logits of a 256-row tile exist only in tensor memory;
// each epilogue thread owns a row and keeps the running maximum and sum of exponentials of its columns, one (max, sum)
// pair per row, column tile and warp goes to the workspace, and a second kernel joins them in a fixed order.
// The target's logit is a dot product of its own, in fp32 by one warp (ce_row_dot: x and W*'s row once more, 2 d elements a
// row), and takes the place of the tensor core's in lse, in the loss and in the gradient. Where the model predicts a row well
// the loss and the target's entry of dl are what is left of exp(l - lse) near 1, and the tensor core's sum is not good enough
// for that: products of one sign are all cut the same way (l = 16.7, d = 4096, sums of 1024 k: 4e-5 low; over all k 1.5e-4),
// so that at 1 - p = 1e-3 the target's row of dW* was 24 % off (0.4 % now). In the join the dot product hides behind
// the product's last tiles.
// Backward: rows without a target have no gradient, so the live rows are packed first and only they go through the three
// products (a batch half of prompt or padding costs half; what such rows hold cannot reach dW*). Then, in pieces of the
// vocabulary, the logits are computed again and leave the chip as the factor both gradients share,
//     P[m, n] = r[m] dl[m, n] in bf16,   dl[m, n] = g[m] (exp(l - lse) - [n = t]),
// except for the target's own entry u[m] = r dl[m, t], which is taken from ce_row_dot and stays fp32 (P is 0 there; in blocks of
// 32 live rows where three targets or more, equal or not, lie within 32 neighbouring classes of a large vocabulary, P has it
// rounded, and u is the rest, which dW* then leaves out):
//     dW*[n, :] = sum_m P[m, n] x[m, :] + sum_{m: t[m] = n} u[m] x[m, :]
//     dx[m, :]  = sum_n P[m, n] W*[n, :] + u[m] W*[t, :] - x[m, :] (r[m]^2 / d) c[m],   c[m] = sum_n dl[m, n] l[m, n]
// (the last term is the norm's own share: dr/dx = -r^3 x / d). The target's entry is most of a row's gradient and would
// pass its rounding on to a whole row of dx and dW*: 0.0024 against 0.0017 relative, output rounding included. That is what
// the rows of dW* of such neighbouring targets get. The other entries are off by at most half a step, 2^-8 of themselves. Over many
// rows or classes of like size that averages out; where one wrong class dominates a row, or few rows make up the batch, it
// stays. Tensor-core speed in both products depends on it. Sums, c and the statistics are fp32.
//
// Measured at 2048 x 4096 x 32000 (each product 537 GFLOP): loss 326 us for the product, 7 and 12 around it; gradient, in two
// pieces, packing 11, P 166 and both gradients' products 338 a piece, dx's last pass 20, together 1.04 ms for one call and
// 1.25 back to back under the power cap (cuBLAS's rate there is 1.42 PFLOP/s: 1.13 ms for the products alone).
// At 517 x 576 x 50257 (a tile of dW* has 8 stages of k): P 34, products 68 us, bound by the L2 and the epilogues.
#pragma once

#include "elementwise.cuh"
#include "pair_gemm.cuh"

namespace fn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float v) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
  return e;
}

// r[m] = 1/sqrt(mean(x[m]^2) + eps), one warp per row. Also zeroes the word `zero` of the kernel that follows (its arrivals, or
// whether it failed).
__global__ void __launch_bounds__(256) k_row_rstd(const uint16_t* __restrict__ x, float* __restrict__ rstd,
                                                  unsigned* __restrict__ zero, int M, int K, float eps) {
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) *zero = 0u;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= M) return;
  const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<size_t>(row) * K);
  float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
  for (int c = lane; c < (K >> 3); c += 32) {
    const uint4 v = __ldcg(src + c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = bf16lo_to_f32(w[e]), b = bf16hi_to_f32(w[e]);
      s0 = fmaf(a, a, s0);
      s1 = fmaf(b, b, s1);
    }
  }
  const float ss = warp_sum(s0 + s1);
  if (lane == 0) rstd[row] = 1.0f / sqrtf(ss / static_cast<float>(K) + eps);
}

// What a target says: a class, nothing (ignore_index), or neither (reported to the host).
__device__ __forceinline__ bool target_is_class(long long t, int V) { return t >= 0 && t < V; }

// x . w of two bf16 rows by a warp in fp32, eight sums a lane, rounded to nearest: within about 2^-24 sqrt(d) of the products'
// magnitudes. The same bits wherever it is taken (lane l adds pieces l, l + 32, ... in order), so that the forward's lse and
// the gradient's logit of a target cancel.
struct CeDot {
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(const uint4& a, const uint4& b) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[2 * e] = fmaf(bf16lo_to_f32(u[e]), bf16lo_to_f32(v[e]), s[2 * e]);
      s[2 * e + 1] = fmaf(bf16hi_to_f32(u[e]), bf16hi_to_f32(v[e]), s[2 * e + 1]);
    }
  }
  __device__ __forceinline__ float total() const {
    return warp_sum(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
  }
};
__device__ __forceinline__ float ce_row_dot(const uint16_t* x, const uint16_t* w, int K, int lane) {
  const uint4* a = reinterpret_cast<const uint4*>(x);
  const uint4* b = reinterpret_cast<const uint4*>(w);
  CeDot dot;
#pragma unroll 4
  for (int c = lane; c < (K >> 3); c += 32) dot.add(__ldcg(a + c), __ldcg(b + c));
  return dot.total();
}

// ---------------------------------------------------------------------------------------------- forward

struct CeFwdParams {
  const float* rstd;
  const long long* targets;
  // [M][kParts column tiles]: running maximum (of log2 e times the logits) and sum of 2^(. - max), the target left out
  float2* part;
};

// A thread's columns of a tile are up to kChunks chunks of 32, shared out among the quarter's warps. HELD: the tile takes
// several accumulations, whose sums so far stay in registers.
template <bool HELD>
struct CeFwdEpi {
  static constexpr int kParts = 4;
  static constexpr int kChunks = 8 / kParts;
  using Params = CeFwdParams;
  float r2;  // r log2(e): the exponentials are powers of two
  long long tgt;
  float held[HELD ? kChunks : 1][32];
  __device__ __forceinline__ CeFwdEpi(const Params& e, const PairGemmParams& p, const PgTile& t, int lane) {
    const int row = t.row0 + lane;
    r2 = row < t.M ? __ldcg(e.rstd + row) * kLog2e : 0.f;
    tgt = row < t.M ? __ldg(e.targets + row) : -1;
    if (HELD) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
#pragma unroll
        for (int j = 0; j < 32; ++j) held[HELD ? i : 0][j] = 0.f;
    }
  }
  __device__ __forceinline__ void run(const Params& e, const PairGemmParams& p, const PgTile& t, int lane) {
    const int row = t.row0 + lane;
    const int c00 = 32 * t.part;
    float m = -INFINITY, s = 0.f;
    if (HELD && t.chunk < t.chunks - 1) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        uint32_t v[2][16];
        if (c00 + 32 * kParts * i >= t.width) continue;
        tmem_ld16(t.t_row + c00 + 32 * kParts * i, v[0]);
        tmem_ld16(t.t_row + c00 + 32 * kParts * i + 16, v[1]);
        tmem_ld_wait();
        reg_fence16(v[0]);
        reg_fence16(v[1]);
#pragma unroll
        for (int j = 0; j < 32; ++j) held[HELD ? i : 0][j] += __uint_as_float(v[j >> 4][j & 15]);
      }
      return;
    }
    // with sums held, 16 columns at a time, which saves registers
    constexpr int kCols = HELD ? 16 : 32;
#pragma unroll(HELD ? kChunks * 2 : 1)
    for (int i = 0; i < kChunks * 32 / kCols; ++i) {
      const int c0 = c00 + 32 * kParts * (i * kCols / 32) + i * kCols % 32;
      if (c0 >= t.width) break;
      float z[kCols];
      {
        uint32_t v[kCols / 16][16];
#pragma unroll
        for (int b = 0; b < kCols / 16; ++b) tmem_ld16(t.t_row + c0 + 16 * b, v[b]);
        tmem_ld_wait();
#pragma unroll
        for (int b = 0; b < kCols / 16; ++b) reg_fence16(v[b]);
#pragma unroll
        for (int j = 0; j < kCols; ++j)
          z[j] = (HELD ? held[HELD ? i * kCols / 32 : 0][HELD ? i * kCols % 32 + j : 0] : 0.f) + __uint_as_float(v[j >> 4][j & 15]);
      }
      const bool edge = c0 + kCols > t.width;  // columns past the vocabulary take no part
      if (edge) {
#pragma unroll
        for (int j = 1; j < kCols; ++j)
          if (c0 + j >= t.width) z[j] = z[0];
      }
      const long long at = tgt - (t.n0 + c0);
      if (at >= 0 && at < kCols) {  // the target joins the row at the end
#pragma unroll
        for (int j = 0; j < kCols; ++j)
          if (at == j) z[j] = -INFINITY;
      }
      float mc = z[0];
#pragma unroll
      for (int j = 1; j < kCols; ++j) mc = fmaxf(mc, z[j]);
      const float mn = fmaxf(m, mc * r2);
      const float base = mn == -INFINITY ? 0.f : mn;  // a row of -inf so far: 2^(-inf) = 0, not NaN
      const uint64_t rr = pack_f32x2(r2, r2), nb = pack_f32x2(-base, -base);
      uint64_t a0 = 0, a1 = 0;
#pragma unroll
      for (int j = 0; j < kCols; j += 4) {
        const float2 q0 = unpack_f32x2(fma_f32x2(pack_f32x2(z[j], z[j + 1]), rr, nb));
        const float2 q1 = unpack_f32x2(fma_f32x2(pack_f32x2(z[j + 2], z[j + 3]), rr, nb));
        float e0 = ex2(q0.x), e1 = ex2(q0.y), e2 = ex2(q1.x), e3 = ex2(q1.y);
        if (edge) {
          if (c0 + j >= t.width) e0 = 0.f;
          if (c0 + j + 1 >= t.width) e1 = 0.f;
          if (c0 + j + 2 >= t.width) e2 = 0.f;
          if (c0 + j + 3 >= t.width) e3 = 0.f;
        }
        a0 = add_f32x2(a0, pack_f32x2(e0, e1));
        a1 = add_f32x2(a1, pack_f32x2(e2, e3));
      }
      const float2 sum = unpack_f32x2(add_f32x2(a0, a1));
      s = s * ex2(m - base) + (sum.x + sum.y);
      m = mn;
    }
    if (row < t.M)
      e.part[static_cast<size_t>(row) * (kParts * p.num_n_tiles) + kParts * t.nt + t.part] = make_float2(m, s);
  }
};

// lse and loss of a row by LANES consecutive lanes: each joins every LANES-th partial pair, then they join in a butterfly (a
// fixed order), and last the target's logit, rstd zt. BATCH pairs of a lane are loaded at once. An ignored row's loss is 0;
// a target t that is neither a class nor ignore_index gives NaN and is reported. Every lane of the warp calls, live or not.
template <int LANES, int BATCH>
__device__ __forceinline__ void ce_join_row(const float2* part, int parts, float rstd, float zt, long long t, float* loss,
                                            float* lse, int row, bool live, int V, long long ignore, int lane) {
  const int sub = lane % LANES;
  const float2* src = part + static_cast<size_t>(live ? row : 0) * parts;
  float m = -INFINITY, s = 0.f;
  auto join = [&](float qm, float qs) {
    const float mn = fmaxf(m, qm);
    const float base = mn == -INFINITY ? 0.f : mn;
    s = s * ex2(m - base) + qs * ex2(qm - base);
    m = mn;
  };
  for (int i0 = sub; i0 < parts; i0 += BATCH * LANES) {
    float2 q[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
      q[k] = live && i0 + k * LANES < parts ? __ldcg(src + i0 + k * LANES) : make_float2(-INFINITY, 0.f);
    // the batch's maximum first: one exponential a pair instead of two
    float mn = m;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) mn = fmaxf(mn, q[k].x);
    const float base = mn == -INFINITY ? 0.f : mn;
    s *= ex2(m - base);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) s = fmaf(q[k].y, ex2(q[k].x - base), s);
    m = mn;
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) join(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o));
  if (sub == 0 && live) {
    const float lt = zt * (rstd * kLog2e);
    if (target_is_class(t, V)) join(lt, 1.0f);
    const float ls = logf(s);
    lse[row] = m * kLn2 + ls;
    if (t == ignore) {
      loss[row] = 0.f;
    } else if (target_is_class(t, V)) {
      loss[row] = fmaf(m - lt, kLn2, ls);  // lse - l_t, without the rounding of lse
    } else {
      loss[row] = __int_as_float(0x7fc00000);
      atomicOr(&g_device_status, kStatusBadTarget);
    }
  }
}

// A warp per row. x, W* and the targets are in place before the product starts (the row statistics' pass waited for them), so
// the target's logit is taken before the wait. A product that gave up (*failed) has left pairs unwritten: NaN then, as the status
// word reports.
__global__ void __launch_bounds__(256) k_ce_join(const float2* __restrict__ part, const float* __restrict__ rstd,
                                                 const uint16_t* __restrict__ x, const uint16_t* __restrict__ W,
                                                 const long long* __restrict__ targets, const unsigned* failed,
                                                 float* __restrict__ loss, float* __restrict__ lse, int M, int K, int V,
                                                 int parts, long long ignore) {
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const long long t = row < M ? __ldcg(targets + row) : ignore;
  const float zt = row < M && target_is_class(t, V)
                       ? ce_row_dot(x + static_cast<size_t>(row) * K, W + static_cast<size_t>(t) * K, K, lane) : 0.f;
  grid_dep_wait();
  grid_dep_launch();
  const unsigned gave_up = __ldcg(failed);  // looked at last: its load runs beside those of the pairs
  ce_join_row<32, 10>(part, parts, row < M ? __ldcg(rstd + row) : 0.f, zt, t, loss, lse, row, row < M, V, ignore, lane);
  if (gave_up != 0u && row < M && lane == 0) loss[row] = lse[row] = __int_as_float(0x7fc00000);
}

// ---------------------------------------------------------------------------------------------- backward

// What the products need of a live row.
struct __align__(16) CeRow {
  float rstd, nlse2, g;  // 1/rms, -lse log2(e), dL/dloss
  int target;
};

// What the other two products and the last kernel need of them.
struct CeLive {
  const int* n_live;
  int* target;  // [live rows]
  float* u;     // r dl of the target's entry, from where P has it less that
  // [32 vocabulary columns of the piece][ld_hits: 32 live rows]: which of these rows have their target among these columns
  // and its entry not in P
  unsigned* hits;
  int ld_hits;
};

constexpr int kCeIgnored = -1, kCeBad = -2;  // in place of a row's rank among the live ones

// Packs the live rows in order: xc[rank] = x[m], rows[rank], the target's entry u[rank] and its share ct[rank] of c / r,
// rank_of[m], and their number. Rows up to the next multiple of 64 are zeroed: dW*'s product runs over whole stages of 64
// rows. A block serves rows_per_block rows, a warp an eighth of them in order; each counts the live rows before its own, from
// the targets. 2048 x 4096: 11.4 us for 33 MB from HBM, latency: one row a warp.
__global__ void __launch_bounds__(256, 2) k_ce_pack(const uint16_t* __restrict__ x, const long long* __restrict__ targets,
                                                    const float* __restrict__ lse, const float* __restrict__ g,
                                                    const uint16_t* __restrict__ W, uint16_t* __restrict__ xc,
                                                    CeRow* __restrict__ rows, int* __restrict__ target,
                                                    float* __restrict__ u, float* __restrict__ ct,
                                                    int* __restrict__ rank_of, int* __restrict__ n_live, int M, int K,
                                                    int V, int rows_per_block, float eps, long long ignore) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ int counts[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto live_at = [&](int m) {
    const long long t = __ldcg(targets + m);
    return t != ignore && target_is_class(t, V);
  };
  const int b0 = static_cast<int>(blockIdx.x) * rows_per_block;
  const int per_warp = rows_per_block >> 3, m0 = b0 + warp * per_warp;
  const int chunks = K >> 3;
  // a row's first kHeld * 256 elements go through registers, and the first 4 * 256 of its target's row of W*; those of the
  // warp's first row are loaded ahead of the count
  constexpr int kHeld = 16;
  uint4 held[kHeld], w[4];
  auto load_w = [&](long long t, int i0) {
    const uint4* wt = reinterpret_cast<const uint4*>(W + static_cast<size_t>(t) * K);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = lane + 32 * (i0 + i) < chunks ? __ldcg(wt + lane + 32 * (i0 + i)) : make_uint4(0u, 0u, 0u, 0u);
  };
  auto load_row = [&](int m, long long t) {
    const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<size_t>(m) * K);
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      held[i] = lane + 32 * i < chunks ? __ldcg(src + lane + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
    if (target_is_class(t, V)) load_w(t, 0);
  };
  long long t = m0 < M ? __ldcg(targets + m0) : ignore;
  if (m0 < M) load_row(m0, t);
  int n = 0;
#pragma unroll 8
  for (int m = threadIdx.x; m < b0; m += 256) n += live_at(m);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) counts[warp] = n;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) base += counts[i];
  auto count = [&](int from, int to) {
    int c = 0;
    for (int m = from + lane; m < to; m += 32) c += live_at(m);
    return __reduce_add_sync(0xffffffffu, c);
  };
  int rank = base + count(b0, min(m0, M));
  long long t_next;
  for (int m = m0; m < min(m0 + per_warp, M); ++m, t = t_next) {
    t_next = m + 1 < M ? __ldcg(targets + m + 1) : ignore;
    const bool live = t != ignore && target_is_class(t, V);
    if (lane == 0) rank_of[m] = live ? rank : t == ignore ? kCeIgnored : kCeBad;
    if (!live) continue;
    const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<size_t>(m) * K);
    const uint4* wt = reinterpret_cast<const uint4*>(W + static_cast<size_t>(t) * K);
    uint4* dst = reinterpret_cast<uint4*>(xc + static_cast<size_t>(rank) * K);
    float s0 = 0.f, s1 = 0.f;
    CeDot dot;
    auto take = [&](const uint4& v) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = bf16lo_to_f32(w[e]), b = bf16hi_to_f32(w[e]);
        s0 = fmaf(a, a, s0);
        s1 = fmaf(b, b, s1);
      }
    };
    if (m != m0) load_row(m, t);
#pragma unroll
    for (int i0 = 0; i0 < kHeld; i0 += 4) {
      if (i0 > 0) load_w(t, i0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4& v = held[i0 + i];
        if (lane + 32 * (i0 + i) < chunks) dst[lane + 32 * (i0 + i)] = v;
        take(v);
        dot.add(v, w[i]);
      }
    }
#pragma unroll 2
    for (int c = lane + 32 * kHeld; c < chunks; c += 32) {
      const uint4 v = __ldcg(src + c), w = __ldcg(wt + c);
      dst[c] = v;
      take(v);
      dot.add(v, w);
    }
    const float ss = warp_sum(s0 + s1), zt = dot.total();
    if (lane == 0) {
      CeRow r;
      r.rstd = 1.0f / sqrtf(ss / static_cast<float>(K) + eps);
      r.nlse2 = -__ldcg(lse + m) * kLog2e;
      r.g = __ldcg(g + m);
      r.target = static_cast<int>(t);
      rows[rank] = r;
      target[rank] = r.target;
      const float ut = r.g * r.rstd * (ex2(fmaf(zt, r.rstd * kLog2e, r.nlse2)) - 1.0f);
      u[rank] = ut;
      ct[rank] = ut * zt;
    }
    ++rank;
  }
  if (blockIdx.x == gridDim.x - 1) {
    const int live = base + count(b0, M);
    if (threadIdx.x == 0) *n_live = live;
    const int end = (live + 63) & ~63;
    for (int r = live + warp; r < end; r += 8) {
      uint4* dst = reinterpret_cast<uint4*>(xc + static_cast<size_t>(r) * K);
      for (int c = lane; c < chunks; c += 32) dst[c] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

struct CeGradParams {
  const CeRow* rows;
  uint16_t* P;     // bf16 [live rows, and up to the next multiple of 64][ldp], this piece's columns
  float* cpart;    // [kParts column tiles][M] partial c without the targets' share, this piece's
  int ldp;         // a multiple of 64: rows of P start on whole 128-byte lines
  int v0;          // first column of the piece within the vocabulary
  int often;       // targets in a block of 32 rows and 32 classes from which on P has them
  CeLive live;
};

struct CeGradEpi {
  static constexpr int kParts = 2;
  using Params = CeGradParams;
  CeRow q;
  __device__ __forceinline__ CeGradEpi(const Params& e, const PairGemmParams& p, const PgTile& t, int lane) {
    const int row = t.row0 + lane;
    q.rstd = q.g = 0.f;
    q.nlse2 = -INFINITY;  // past the live rows every exponential is 0
    q.target = -1;
    if (row < t.M) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(e.rows + row));
      q.rstd = v.x, q.nlse2 = v.y, q.g = v.z, q.target = __float_as_int(v.w);
    }
  }
  __device__ __forceinline__ void run(const Params& e, const PairGemmParams& p, const PgTile& t, int lane) {
    const int row = t.row0 + lane;
    const float r2 = q.rstd * kLog2e, gr = q.g * q.rstd;
    const uint64_t rr = pack_f32x2(r2, r2), nl = pack_f32x2(q.nlse2, q.nlse2), gg = pack_f32x2(gr, gr);
    uint64_t c2 = 0;  // sum of exp(l - lse) z; c = g r times it
    float ct = 0.f;   // the target's share of that, negative: c takes it from ce_row_dot
    const int t0 = q.target - (e.v0 + t.n0);  // the target's column in this tile, if it has it
    for (int ch = t.part; ch * 32 < t.width; ch += kParts) {
      const int c0 = ch * 32;
      uint32_t v[2][16];
      tmem_ld16(t.t_row + c0, v[0]);
      tmem_ld16(t.t_row + c0 + 16, v[1]);
      tmem_ld_wait();
      reg_fence16(v[0]);
      reg_fence16(v[1]);
      const bool edge = t.row0 + 32 > t.M || c0 + 32 > t.width;
      if (edge) {  // whatever lies past the live rows or the vocabulary takes no part
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (row >= t.M || c0 + j >= t.width) v[j >> 4][j & 15] = 0u;
      }
      uint32_t w[16];
      float2 o[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint64_t z = pack_f32x2(__uint_as_float(v[j >> 3][2 * (j & 7)]), __uint_as_float(v[j >> 3][2 * (j & 7) + 1]));
        const float2 a = unpack_f32x2(fma_f32x2(z, rr, nl));
        const uint64_t ex = pack_f32x2(ex2(a.x), ex2(a.y));
        c2 = fma_f32x2(ex, z, c2);
        o[j] = unpack_f32x2(mul_f32x2(ex, gg));
      }
      if (edge) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c0 + j >= t.width) {
            if (j & 1) o[j >> 1].y = 0.f; else o[j >> 1].x = 0.f;
          }
      }
      const int at = t0 - c0;
      const bool hit = row < t.M && at >= 0 && at < 32 && c0 + at < t.width;
      const unsigned hits = __ballot_sync(0xffffffffu, hit);
      // `often` rows of the block or more, of one frequent class or of several next to each other (ids in order of frequency,
      // as vocabularies have them): dW* takes their entries from P, with one rounding each, so that no warp of its epilogue
      // has more than two rows in 32 to add by itself. Counting only rows of one class and keeping the first two others of
      // each block exact takes 420 us for 2048 x 1024 x 32000 with targets of frequency 1 / id, 340 so (2048 x 1024 x 32000 with a
      // tenth of the rows, or all, of one class: 341 and 318 us; 496 and 2323 if all are added there; 326 with none).
      const bool often = __popc(hits) >= e.often;
      if (lane == 0) e.live.hits[static_cast<size_t>((t.n0 + c0) >> 5) * e.live.ld_hits + (t.row0 >> 5)] = often ? 0u : hits;
      if (hit) {  // the target's entry: kept in fp32, 0 in P, or what its rounding in P leaves of it
        float z = 0.f, in_p = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (at == j) z = __uint_as_float(v[j >> 4][j & 15]);
        ct = -z * ex2(fmaf(z, r2, q.nlse2));
        if (often) {
          const float u = __ldcg(e.live.u + row);
          in_p = bf16lo_to_f32(pack_bf16x2(u, 0.f) & 0xFFFFu);
          e.live.u[row] = u - in_p;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (at == j) {
            if (j & 1) o[j >> 1].y = in_p; else o[j >> 1].x = in_p;
          }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(o[j].x, o[j].y);
#pragma unroll
      for (int j = 0; j < 4; ++j) pg_put(t.stage, lane, j, make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
      // zeros up to the end of the stage of 64 rows that dW*'s product reads
      pg_flush(t.stage, lane, e.P, static_cast<size_t>(e.ldp) * 2, t.row0, (t.M + 63) & ~63, 2ll * (t.n0 + c0), 2ll * e.ldp);
    }
    const float2 cs = unpack_f32x2(c2);
    if (row < t.M) e.cpart[static_cast<size_t>(kParts * t.nt + t.part) * p.M + row] = gr * ((cs.x + cs.y) + ct);
  }
};

// dW*: the product plus the target entries' share, rounded to bf16 once. Of a warp's 32 vocabulary rows few are a target:
// while the MMAs run it lists the live rows that have one of them (from the masks that P's epilogue left, 4 bytes per 32
// live rows), lane k the k-th. They are added in their order, eight at a time: the lanes load the chunk's 32 columns of
// u x (for the first eight one chunk ahead) and pass them through the staging buffer to the lane whose row it is. A warp
// with more than 32 hits lists the further ones again in every chunk.
struct CeDwParams {
  CeLive live;
  const uint16_t* xc;  // [live rows][ldy]
  uint16_t* y;
  int ldy;
  int v0;
};
struct CeDwHits {
  int n;     // how many, the same in every lane
  int next;  // first live row not looked at
  int r;     // lane k: live row of hit k, its vocabulary row within the warp's, its u
  int row;
  float u;
};
struct CeDwEpi {
  static constexpr int kParts = 2;
  using Params = CeDwParams;
  int base, live;  // first vocabulary row of the warp; live rows
  int slab;        // the warp's row of the masks
  CeDwHits first;
  float val[8];  // of the first eight hits, for the chunk to come

  __device__ __forceinline__ CeDwHits look(const Params& e, int from, int lane) const {
    CeDwHits h = {0, live, 0, 0, 0.f};
    const unsigned* masks = e.live.hits + static_cast<size_t>(slab) * e.live.ld_hits;
    const int words = (live + 31) >> 5;
    for (int g0 = from >> 5; g0 < words; g0 += 128) {
      unsigned w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = g0 + 32 * i + lane < words ? __ldcg(masks + g0 + 32 * i + lane) : 0u;
      if (lane == 0 && g0 == from >> 5) w[0] &= 0xffffffffu << (from & 31);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        for (unsigned some = __ballot_sync(0xffffffffu, w[i] != 0); some != 0; some &= some - 1) {
          const int src = __ffs(some) - 1;
          for (unsigned hits = __shfl_sync(0xffffffffu, w[i], src); hits != 0; hits &= hits - 1) {
            const int r = 32 * (g0 + 32 * i + src) + __ffs(hits) - 1;
            if (h.n == 32) {
              h.next = r;
              goto done;
            }
            if (lane == h.n) h.r = r;
            ++h.n;
          }
        }
      }
    }
  done:
    if (lane < h.n) {
      h.row = __ldcg(e.live.target + h.r) - base;
      h.u = __ldcg(e.live.u + h.r);
    }
    return h;
  }
  // u x of hits k0 .. k0+7 at the lane's column
  __device__ __forceinline__ void fetch(const Params& e, const CeDwHits& h, int k0, int col, int N) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = __shfl_sync(0xffffffffu, h.r, (k0 + k) & 31);
      const float u = __shfl_sync(0xffffffffu, h.u, (k0 + k) & 31);
      val[k] = k0 + k < h.n && col < N ? u * bf16lo_to_f32(__ldg(e.xc + static_cast<size_t>(r) * e.ldy + col)) : 0.f;
    }
  }
  // Slot k of the staging buffer holds hit k0 + k: 32 floats, piece j at (j + k) % 8.
  __device__ __forceinline__ void stage(const PgTile& t, int lane) const {
    float* slots = reinterpret_cast<float*>(t.stage);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) slots[k * 32 + (((lane >> 2) + k) & 7) * 4 + (lane & 3)] = val[k];
    __syncwarp();
  }
  __device__ __forceinline__ void add(const CeDwHits& h, int k0, const PgTile& t, int lane, uint32_t (&v)[2][16]) const {
    const float* slots = reinterpret_cast<const float*>(t.stage);
    for (int k = 0; k0 + k < h.n && k < 8; ++k) {
      if (__shfl_sync(0xffffffffu, h.row, k0 + k) != lane) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 a = *reinterpret_cast<const float4*>(slots + k * 32 + ((j + k) & 7) * 4);
        uint32_t* w = &v[j >> 2][4 * (j & 3)];
        w[0] = __float_as_uint(__uint_as_float(w[0]) + a.x);
        w[1] = __float_as_uint(__uint_as_float(w[1]) + a.y);
        w[2] = __float_as_uint(__uint_as_float(w[2]) + a.z);
        w[3] = __float_as_uint(__uint_as_float(w[3]) + a.w);
      }
    }
    __syncwarp();
  }

  __device__ __forceinline__ CeDwEpi(const Params& e, const PairGemmParams& p, const PgTile& t, int lane) {
    base = e.v0 + t.row0;
    slab = t.row0 >> 5;
    live = t.row0 < t.M ? __ldcg(e.live.n_live) : 0;
    first = look(e, 0, lane);
    if (first.n > 0) fetch(e, first, 0, t.n0 + 32 * t.part + lane, p.N);
  }
  __device__ __forceinline__ void run(const Params& e, const PairGemmParams& p, const PgTile& t, int lane) {
    for (int ch = t.part; ch * 32 < t.width; ch += kParts) {
      uint32_t v[2][16];
      tmem_ld16(t.t_row + ch * 32, v[0]);
      tmem_ld16(t.t_row + ch * 32 + 16, v[1]);
      const int col = t.n0 + ch * 32 + lane;
      if (first.n > 0) {
        stage(t, lane);
        if (first.n <= 8) fetch(e, first, 0, col + 32 * kParts, p.N);
      }
      tmem_ld_wait();
      reg_fence16(v[0]);
      reg_fence16(v[1]);
      if (t.empty) {  // no live rows
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j >> 4][j & 15] = 0u;
      }
      if (first.n > 0) {
        add(first, 0, t, lane, v);
        for (int k0 = 8; k0 < first.n; k0 += 8) {
          fetch(e, first, k0, col, p.N);
          stage(t, lane);
          add(first, k0, t, lane, v);
        }
        for (int from = first.next; from < live;) {
          const CeDwHits h = look(e, from, lane);
          for (int k0 = 0; k0 < h.n; k0 += 8) {
            fetch(e, h, k0, col, p.N);
            stage(t, lane);
            add(h, k0, t, lane, v);
          }
          from = h.next;
        }
        if (first.n > 8) fetch(e, first, 0, col + 32 * kParts, p.N);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t* w = &v[j >> 1][8 * (j & 1)];
        pg_put(t.stage, lane, j,
               make_uint4(pack_bf16x2(__uint_as_float(w[0]), __uint_as_float(w[1])),
                          pack_bf16x2(__uint_as_float(w[2]), __uint_as_float(w[3])),
                          pack_bf16x2(__uint_as_float(w[4]), __uint_as_float(w[5])),
                          pack_bf16x2(__uint_as_float(w[6]), __uint_as_float(w[7]))));
      }
      pg_flush(t.stage, lane, e.y, static_cast<size_t>(e.ldy) * 2, t.row0, t.M, 2ll * (t.n0 + ch * 32), 2ll * e.ldy);
    }
  }
};

// fp32 sums, one plane per K range: dx's over the pieces of the vocabulary (the first piece writes, later ones add), and
// dW*'s where the vocabulary is small (k_ce_dw).
struct CeDxParams {
  float* acc;  // [K ranges][M][ld]
  int ld;      // a multiple of 8
  int add;
};
struct CeDxEpi {
  static constexpr int kParts = 2;
  using Params = CeDxParams;
  __device__ __forceinline__ CeDxEpi(const Params&, const PairGemmParams&, const PgTile&, int) {}
  __device__ __forceinline__ void run(const Params& e, const PairGemmParams& p, const PgTile& t, int lane) {
    float* plane = e.acc + static_cast<size_t>(t.kz) * p.M * e.ld;
    for (int ch = t.part; ch * 16 < t.width; ch += kParts) {
      uint32_t v[16];
      tmem_ld16(t.t_row + ch * 16, v);
      tmem_ld_wait();
      reg_fence16(v);
      if (t.empty) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0u;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) pg_put(t.stage, lane, j, make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
      __syncwarp();
      const int seg = lane & 3, col = t.n0 + ch * 16 + 4 * seg;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = 8 * i + (lane >> 2), row = t.row0 + rr;
        float4 s = *reinterpret_cast<const float4*>(t.stage + rr * 64 + (((seg ^ (rr >> 1)) & 3) << 4));
        if (row < t.M && col < e.ld) {
          float4* dst = reinterpret_cast<float4*>(plane + static_cast<size_t>(row) * e.ld + col);
          if (e.add) {
            const float4 old = __ldcg(dst);
            s = make_float4(s.x + old.x, s.y + old.y, s.z + old.z, s.w + old.w);
          }
          __stcg(dst, s);
        }
      }
      __syncwarp();
    }
  }
};

// dW*[n, :] = sum of the planes + sum over the live rows m with t[m] = n of u[m] x[m, :], one block per class. Used where
// the vocabulary is small: 32 classes then have so many rows that one warp's list of them would take longer than the
// tile's MMAs (the epilogue's way took 147 us at 2167 x 280 x 602, and 268 at 4096 x 64 x 128, where the one tile of dW*
// had to run through all rows besides), and planes are cheap. The block looks through 2048 targets at a time, lists its
// own in order, and its threads share out columns (8 each) and, where there are fewer column groups than threads, rows.
__global__ void __launch_bounds__(256) k_ce_dw(const float* __restrict__ acc, const CeLive live, const uint16_t* __restrict__ xc,
                                               uint16_t* __restrict__ dW, int N, int K, int planes, int v0) {
  __shared__ int list[2048];
  __shared__ int counts[8];
  __shared__ float part[256 * 8];
  grid_dep_wait();
  grid_dep_launch();
  const int n = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = __ldcg(live.n_live), chunks = K >> 3;
  const int width = min(chunks, 256), groups = 256 / width;  // column groups side by side, shares of the rows
  const int col = threadIdx.x % width, share = threadIdx.x / width;
  for (int c0 = 0; c0 < chunks; c0 += width) {
    const int c = c0 + col;
    float a[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = 0.f;
    for (int r0 = 0; r0 < rows; r0 += 2048) {
      int t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + 256 * warp + 32 * i + lane;
        t[i] = r < rows ? __ldcg(live.target + r) : -1;
      }
      unsigned hit[8];
      int mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        hit[i] = __ballot_sync(0xffffffffu, t[i] == v0 + n);
        mine += __popc(hit[i]);
      }
      if (lane == 0) counts[warp] = mine;
      __syncthreads();
      int at = 0, total = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w < warp) at += counts[w];
        total += counts[w];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (hit[i] >> lane & 1u) list[at + __popc(hit[i] & ((1u << lane) - 1u))] = r0 + 256 * warp + 32 * i + lane;
        at += __popc(hit[i]);
      }
      __syncthreads();
      if (share < groups && c < chunks) {
#pragma unroll 4
        for (int k = share; k < total; k += groups) {
          const int r = list[k];
          const float u = __ldcg(live.u + r);
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(xc + static_cast<size_t>(r) * K) + c);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[2 * e] = fmaf(u, bf16lo_to_f32(w[e]), a[2 * e]);
            a[2 * e + 1] = fmaf(u, bf16hi_to_f32(w[e]), a[2 * e + 1]);
          }
        }
      }
    }
    if (groups > 1) {
#pragma unroll
      for (int e = 0; e < 8; ++e) part[threadIdx.x * 8 + e] = a[e];
      __syncthreads();
    }
    if (share == 0 && c < chunks) {
      for (int g = 1; g < groups; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] += part[(g * width + col) * 8 + e];
      for (int z = 0; z < planes; ++z) {
        const float4* src = reinterpret_cast<const float4*>(acc + (static_cast<size_t>(z) * N + n) * K) + 2 * c;
        const float4 p = __ldcg(src), q = __ldcg(src + 1);
        a[0] += p.x, a[1] += p.y, a[2] += p.z, a[3] += p.w, a[4] += q.x, a[5] += q.y, a[6] += q.z, a[7] += q.w;
      }
      reinterpret_cast<uint4*>(dW + static_cast<size_t>(n) * K)[c] =
          make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
    }
    __syncthreads();  // list, counts and part are used again
  }
}

// dx[m, :] = sum of the planes + u[m] W*[t, :] - x[m, :] (r^2 / d) c[m], LPR threads per row; planes and partial sums c by
// the row's rank among the live ones, in a fixed order. A thread's first 16 columns are on their way while c is summed.
template <int LPR>
__global__ void __launch_bounds__(256) k_ce_dx(const float* __restrict__ acc, const float* __restrict__ cpart,
                                               const CeRow* __restrict__ rows, const float* __restrict__ u,
                                               const float* __restrict__ ct,
                                               const uint16_t* __restrict__ x, const uint16_t* __restrict__ W,
                                               const int* __restrict__ rank_of, uint16_t* __restrict__ dx, int M, int K,
                                               int planes, int parts) {
  __shared__ float red[8];
  grid_dep_wait();
  grid_dep_launch();
  const int row = blockIdx.x * (256 / LPR) + threadIdx.x / LPR, sub = threadIdx.x % LPR;
  if (row >= M) return;  // whole warps; with a block per row there is no such block
  const int rank = __ldcg(rank_of + row), chunks = K >> 3;
  uint4* dst = reinterpret_cast<uint4*>(dx + static_cast<size_t>(row) * K);
  if (rank < 0) {
    const bool bad = rank == kCeBad;
    const uint32_t w = bad ? 0x7FC07FC0u : 0u;
    for (int c = sub; c < chunks; c += LPR) dst[c] = make_uint4(w, w, w, w);
    if (bad && sub == 0) atomicOr(&g_device_status, kStatusBadTarget);
    return;
  }
  const float4 meta = __ldcg(reinterpret_cast<const float4*>(rows + rank));
  const float r = meta.x, ut = __ldcg(u + rank), c_t = __ldcg(ct + rank);
  const uint4* wr = reinterpret_cast<const uint4*>(W + static_cast<size_t>(__float_as_int(meta.w)) * K);
  const uint4* xr = reinterpret_cast<const uint4*>(x + static_cast<size_t>(row) * K);
  const float4* ar = reinterpret_cast<const float4*>(acc + static_cast<size_t>(rank) * K);
  const size_t plane = static_cast<size_t>(M) * K / 4;
  constexpr int kAhead = 2;
  float4 a[kAhead], b[kAhead];
  uint4 v[kAhead], w[kAhead];
  auto load = [&](int i0) {
#pragma unroll
    for (int h = 0; h < kAhead; ++h) {
      const int i = i0 + h * LPR;
      if (i >= chunks) break;
      a[h] = __ldcg(ar + 2 * i), b[h] = __ldcg(ar + 2 * i + 1);
      v[h] = __ldcg(xr + i), w[h] = __ldcg(wr + i);
    }
  };
  load(sub);
  float c = 0.f;
#pragma unroll 4
  for (int i = sub; i < parts; i += LPR) c += __ldcg(cpart + static_cast<size_t>(i) * M + rank);
  c = warp_sum(c);
  if (LPR > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = c;
    __syncthreads();
    c = ((red[0] + red[1]) + (red[2] + red[3])) + ((red[4] + red[5]) + (red[6] + red[7]));
  }
  const float k = r * r / static_cast<float>(K) * (c + c_t);
  for (int i0 = sub; i0 < chunks; i0 += kAhead * LPR) {
    if (i0 != sub) load(i0);
#pragma unroll
    for (int h = 0; h < kAhead; ++h) {
      const int i = i0 + h * LPR;
      if (i >= chunks) break;
      float s[8] = {a[h].x, a[h].y, a[h].z, a[h].w, b[h].x, b[h].y, b[h].z, b[h].w};
#pragma unroll 4
      for (int z = 1; z < planes; ++z) {
        const float4 p = __ldcg(ar + z * plane + 2 * i), q = __ldcg(ar + z * plane + 2 * i + 1);
        s[0] += p.x, s[1] += p.y, s[2] += p.z, s[3] += p.w, s[4] += q.x, s[5] += q.y, s[6] += q.z, s[7] += q.w;
      }
      const uint32_t ww[4] = {w[h].x, w[h].y, w[h].z, w[h].w}, vv[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = pack_bf16x2(fmaf(-k, bf16lo_to_f32(vv[e]), fmaf(ut, bf16lo_to_f32(ww[e]), s[2 * e])),
                           fmaf(-k, bf16hi_to_f32(vv[e]), fmaf(ut, bf16hi_to_f32(ww[e]), s[2 * e + 1])));
      dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

}  // namespace fn
