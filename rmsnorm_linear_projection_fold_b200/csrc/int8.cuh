// int8.cuh — the W8A8 projection: 8-bit integer weights with one scale per output channel, activations quantized
// on the fly to 8-bit integers with one scale per row, and the product between them exact in int32.
//
//     a[m]   = max_k |x[m, k]|,   q[m, k] = round(127 x[m, k] / a[m])        (ties to even; 0 for a row of zeros)
//     rho[m] = a[m] / 127 / sqrt(mean_k x[m, k]^2 + eps)                      (no norm: a[m] / 127)
//     s[n]   = max_k |g[k] W[k, n]| / 127,   Q[n, k] = round(g[k] W[k, n] / s[n])   (s = 1 for a channel of zeros, NaN for
//                                                                                   one that is not finite)
//     y[m, n] = rho[m] s[n] sum_k q[m, k] Q[n, k]
// The deferred normalisation of "FlashNorm: Fast Normalization for Transformers" (Abstract, item ii) costs nothing
// here: 1/rms is a row scalar, and so is the scale that any per-token quantization multiplies the product with.
//
// A call is a row pass (codes and rho, 3 bytes moved per element of x) and a product on kind::i8 tensor cores: CTA
// pairs (pair_gemm.cuh) above 16 rows. Up to 16 rows it is one launch that quantizes for itself
// (decode_int8_cluster.cuh), or, where a K range's codes do not fit on chip, the row pass and decode_int8.cuh.
//
// Measured: 2048 x 4096 -> 2 x 11008 (GLU), row pass 10.3 us, product 117 us (3.2 POP/s; back to back 144 us in all under
// the power cap); 333 x 4096 -> 4096 fp32, 4.5 and 15.8 us, the latter 32 stages of load latency on 64 tiles.
#pragma once

#include "elementwise.cuh"
#include "pair_gemm.cuh"

namespace fn {

// ---------------------------------------------------------------------------------------------- weights (offline)

// Offline, and not near its floor: 4096 x 12288 takes 172 us for 151 MB (576 x 960 10, 4096 x 22016 GLU 205; the bf16 fold 41, 2
// and 73), most of it the scales' serial loop over k.

// s[row] of every output channel: 32 channels per block, eight k slices of each joined in shared memory. For GLU the
// channel's row is the interleaved one (fold_dst_row). Magnitudes are compared as bits, where NaN orders above infinity and
// both above every number: a channel that holds either gets the scale NaN (and, x / NaN being NaN, zero codes), so that it
// shows in what is computed from it, as a row of x with such a value does.
__global__ void __launch_bounds__(256) k_int8_scales(const uint16_t* W, const uint16_t* g,
                                                     float* scales, int d, int N, int glu) {
  __shared__ uint32_t part[8][32];
  grid_dep_wait();
  const int n = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5;
  uint32_t amax = 0;
  if (n < N)
    for (int k = sl; k < d; k += 8)
      amax = max(amax, __float_as_uint(bf16lo_to_f32(g[k]) * bf16lo_to_f32(W[static_cast<size_t>(k) * N + n])) & 0x7FFFFFFFu);
  part[sl][threadIdx.x & 31] = amax;
  __syncthreads();
  if (sl == 0 && n < N) {
    for (int i = 1; i < 8; ++i) amax = max(amax, part[i][threadIdx.x]);
    const float a = __uint_as_float(amax >= 0x7F800000u ? 0x7FC00000u : amax);
    scales[fold_dst_row(n, N / 2, glu != 0)] = a == 0.0f ? 1.0f : __fdiv_rn(a, 127.0f);
  }
}

// The codes, K-major: one 64 x 64 tile of W per block through shared memory, as k_fold does. d % 16 == 0, N % 8 == 0.
__global__ void __launch_bounds__(256) k_fold_int8(const uint16_t* W, const uint16_t* g,
                                                   const float* scales, int8_t* Q, int d,
                                                   int N, int glu) {
  __shared__ float tile[kFoldTile][kFoldTile + 1];  // [n][k]
  const int k0 = blockIdx.y * kFoldTile, n0 = blockIdx.x * kFoldTile;
  grid_dep_wait();
  for (int i = threadIdx.x; i < kFoldTile * 8; i += 256) {
    const int kk = i >> 3, ch = i & 7, k = k0 + kk, n = n0 + ch * 8;
    if (k < d && n < N) {
      const uint4 v = *reinterpret_cast<const uint4*>(W + static_cast<size_t>(k) * N + n);
      const float gk = bf16lo_to_f32(g[k]);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        tile[ch * 8 + 2 * e][kk] = gk * bf16lo_to_f32(w[e]);  // exact: a bf16 x bf16 product fits fp32
        tile[ch * 8 + 2 * e + 1][kk] = gk * bf16hi_to_f32(w[e]);
      }
    }
  }
  __syncthreads();
  {  // one 16-byte store of 16 codes per thread
    const int nn = threadIdx.x >> 2, ch = threadIdx.x & 3, n = n0 + nn, k = k0 + ch * 16;
    if (n < N && k < d) {
      const int row = fold_dst_row(n, N / 2, glu != 0);
      const float s = scales[row];
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int q = max(-127, min(127, __float2int_rn(__fdiv_rn(tile[nn][ch * 16 + 4 * e + j], s))));
          w[e] |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * j);
        }
      }
      *reinterpret_cast<uint4*>(Q + static_cast<size_t>(row) * d + k) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ---------------------------------------------------------------------------------------------- the row pass

// Largest magnitude (two 16-bit ones: they order as unsigned bits, NaN above infinity) and sum of squares (two halves) so
// far.
__device__ __forceinline__ void int8_take(const uint4& v, uint64_t& ss, uint32_t& amax) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint64_t x = pack_f32x2(bf16lo_to_f32(w[e]), bf16hi_to_f32(w[e]));
    ss = fma_f32x2(x, x, ss);
    amax = __vmaxu2(amax, w[e] & 0x7FFF7FFFu);
  }
}

// A row's scale, and the codes it gives: 127 x / a to the nearest integer, ties to even, decided exactly. A row with an
// infinity or a NaN has zero codes and rho = NaN.
struct Int8Row {
  float a, inv, up, rho;
  bool finite;
  __device__ __forceinline__ Int8Row(uint32_t magnitude, float ss, int K, float eps, int norm) {
    finite = magnitude < 0x7F80u;
    a = __uint_as_float(magnitude << 16);
    float r = __fdiv_rn(a, 127.0f);
    if (norm) r *= 1.0f / sqrtf(ss / static_cast<float>(K) + eps);
    rho = finite ? r : __int_as_float(0x7fc00000);
    // rows near the ends of the exponent range are scaled by a power of two (exact), so that neither 127 / a nor 127 x
    // overflows
    up = a < 1e-30f ? 0x1p100f : a > 1e30f ? 0x1p-20f : 1.0f;
    a *= up;
    inv = finite && a > 0.f ? __fdiv_rn(127.0f, a) : 0.0f;
  }
  // Eight codes. x inv is within 2^-16 of the true quotient (inv is rounded once); adding 1.5 * 2^23 in the same fma rounds
  // it to the nearest integer n, which the sum's low byte then holds. What is left of x inv shows how near to a tie it is;
  // only there can n be wrong, and 127 x - n a decides: 127 x and n a have 16 bits, so the fma is exact.
  __device__ __forceinline__ uint2 codes(const uint4& v) const {
    if (!finite) return make_uint2(0u, 0u);
    constexpr float kMagic = 12582912.0f;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const uint64_t ii = pack_f32x2(inv, inv), mm = pack_f32x2(kMagic, kMagic), neg = pack_f32x2(-1.0f, -1.0f);
    uint64_t x[4];
    uint32_t t[8];
    float far = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = pack_f32x2(bf16lo_to_f32(w[e]), bf16hi_to_f32(w[e]));
    if (up != 1.0f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = mul_f32x2(x[e], pack_f32x2(up, up));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t r2 = fma_f32x2(x[e], ii, mm);
      const float2 f = unpack_f32x2(fma_f32x2(x[e], ii, fma_f32x2(r2, neg, mm))), r = unpack_f32x2(r2);
      far = fmaxf(far, fmaxf(fabsf(f.x), fabsf(f.y)));
      t[2 * e] = __float_as_uint(r.x);
      t[2 * e + 1] = __float_as_uint(r.y);
    }
    if (far > 0.5f - 1.0f / 8192.0f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 xx = unpack_f32x2(x[e >> 1]);
        const float n = __uint_as_float(t[e]) - kMagic, rest = fmaf(-n, a, 127.0f * (e & 1 ? xx.y : xx.x));
        const float off = 2.0f * fabsf(rest);
        if (off > a || (off == a && (t[e] & 1u))) t[e] = rest > 0.f ? t[e] + 1 : t[e] - 1;
      }
    }
    uint2 o;
    o.x = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
    o.y = __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410);
    return o;
  }
};

// LPR threads per row, 256 / LPR rows per block; a thread keeps up to 4 x 8 elements of its row in registers, and a
// longer row's remainder is read a second time. x is read once, so past the L1, here and in the other row passes. What the
// kernel before may have written is read behind griddepcontrol.wait, which makes it visible to coherent loads; this kernel starts
// before that one ends, so such data is not constant for its lifetime and never read through the non-coherent path (__ldg).
// Also zeroes the `nzero` words at `zero`, the arrival
// counters of a decode kernel that follows.
// Bound: instruction issue before HBM (2048 x 4096: 25 MB in 10.3 us, launch included; with a conversion and a check per
// code, 14 us). More blocks per SM with fewer registers were slower (11 to 16 us).
template <int LPR>
__global__ void __launch_bounds__(256) k_int8_rows(const uint16_t* __restrict__ x, int8_t* __restrict__ xq,
                                                   float* __restrict__ rho, int M, int K, float eps, int norm,
                                                   unsigned* __restrict__ zero, int nzero) {
  constexpr int kHeld = 4;
  constexpr int kWarps = LPR / 32;  // warps per row
  __shared__ float red_s[8];
  __shared__ uint32_t red_a[8];
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < nzero; i += 256) zero[i] = 0u;
  const int sub = threadIdx.x % LPR, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  const bool live = row < M;
  const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<size_t>(live ? row : 0) * K);
  const int chunks = live ? K >> 3 : 0;
  uint4 held[kHeld];
  uint64_t s2 = 0;
  uint32_t amax = 0;
  auto take = [&](const uint4& v) { int8_take(v, s2, amax); };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = sub + i * LPR;
    held[i] = c < chunks ? __ldcg(src + c) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i) take(held[i]);
  for (int c = sub + kHeld * LPR; c < chunks; c += LPR) take(__ldcg(src + c));
  uint32_t am = max(amax & 0xFFFFu, amax >> 16);
  const float2 halves = unpack_f32x2(s2);
  float ss = halves.x + halves.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
  }
  if (kWarps > 1) {
    if ((threadIdx.x & 31) == 0) {
      red_s[warp] = ss;
      red_a[warp] = am;
    }
    __syncthreads();
    const int w0 = warp / kWarps * kWarps;
    ss = red_s[w0];
    am = red_a[w0];
    for (int i = 1; i < kWarps; ++i) {
      ss += red_s[w0 + i];
      am = max(am, red_a[w0 + i]);
    }
  }
  if (!live) return;
  const Int8Row q(am, ss, K, eps, norm);
  if (sub == 0) rho[row] = q.rho;
  uint2* dst = reinterpret_cast<uint2*>(xq + static_cast<size_t>(row) * K);
  auto put = [&](int c, const uint4& v) { dst[c] = q.codes(v); };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = sub + i * LPR;
    if (c < chunks) put(c, held[i]);
  }
  for (int c = sub + kHeld * LPR; c < chunks; c += LPR) put(c, __ldcg(src + c));
}

// ---------------------------------------------------------------------------------------------- epilogues

// silu(g) u with the SFU's exp2 and reciprocal (relative error about 1e-6); g -> -inf gives -0.
__device__ __forceinline__ float int8_swiglu(float g, float u) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-g * 1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
  return g * s * u;
}

struct Int8EpiParams {
  void* y;            // [M][n_out]
  const float* rho;   // [M]
  const float* scale;  // [rows of Q]
  int n_out;
};

// y = rho s acc, or for GLU silu(rho s_g acc_g) (rho s_u acc_u) with gate and up interleaved in blocks of 16 columns.
template <bool GLU, bool OUT_F32>
struct Int8Epi {
  static constexpr int kParts = 2;
  using Params = Int8EpiParams;
  float rho;
  __device__ __forceinline__ Int8Epi(const Params& e, const PairGemmParams& p, const PgTile& t, int lane) {
    rho = t.row0 + lane < t.M ? __ldcg(e.rho + t.row0 + lane) : 0.f;
  }
  __device__ __forceinline__ void run(const Params& e, const PairGemmParams& p, const PgTile& t, int lane) {
    constexpr int kOut = OUT_F32 ? 16 : 32;      // outputs of a staged block (64 bytes of a row)
    constexpr int kAcc = GLU ? 2 * kOut : kOut;  // its accumulator columns
    constexpr int kEsz = OUT_F32 ? 4 : 2;
    for (int ch = t.part; ch * kAcc < t.width; ch += kParts) {
      const int c0 = ch * kAcc;
      uint32_t v[kAcc / 16][16];
#pragma unroll
      for (int b = 0; b < kAcc / 16; ++b) tmem_ld16(t.t_row + c0 + 16 * b, v[b]);
      tmem_ld_wait();
#pragma unroll
      for (int b = 0; b < kAcc / 16; ++b) reg_fence16(v[b]);
      const float4* sc = reinterpret_cast<const float4*>(e.scale + t.n0 + c0);
#pragma unroll
      for (int b = 0; b < kAcc / 16; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // N % 8 == 0: a group of four channels is wholly inside or wholly outside
          const float4 s4 = c0 + 16 * b + 4 * j < t.width ? __ldg(sc + 4 * b + j) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[b][4 * j] = __float_as_uint(static_cast<float>(static_cast<int>(v[b][4 * j])) * rho * s4.x);
          v[b][4 * j + 1] = __float_as_uint(static_cast<float>(static_cast<int>(v[b][4 * j + 1])) * rho * s4.y);
          v[b][4 * j + 2] = __float_as_uint(static_cast<float>(static_cast<int>(v[b][4 * j + 2])) * rho * s4.z);
          v[b][4 * j + 3] = __float_as_uint(static_cast<float>(static_cast<int>(v[b][4 * j + 3])) * rho * s4.w);
        }
      float o[kOut];
#pragma unroll
      for (int j = 0; j < kOut; ++j) {
        if constexpr (GLU)
          o[j] = int8_swiglu(__uint_as_float(v[2 * (j / 16)][j & 15]), __uint_as_float(v[2 * (j / 16) + 1][j & 15]));
        else
          o[j] = __uint_as_float(v[j / 16][j & 15]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (OUT_F32)
          pg_put(t.stage, lane, j, make_uint4(__float_as_uint(o[4 * j]), __float_as_uint(o[4 * j + 1]),
                                              __float_as_uint(o[4 * j + 2]), __float_as_uint(o[4 * j + 3])));
        else
          pg_put(t.stage, lane, j, make_uint4(pack_bf16x2(o[8 * j], o[8 * j + 1]), pack_bf16x2(o[8 * j + 2], o[8 * j + 3]),
                                              pack_bf16x2(o[8 * j + 4], o[8 * j + 5]), pack_bf16x2(o[8 * j + 6], o[8 * j + 7])));
      }
      const int oc0 = GLU ? (t.n0 + c0) / 2 : t.n0 + c0;
      pg_flush(t.stage, lane, e.y, static_cast<size_t>(e.n_out) * kEsz, t.row0, t.M, static_cast<long long>(oc0) * kEsz,
               static_cast<long long>(e.n_out) * kEsz);
    }
  }
};

}  // namespace fn
