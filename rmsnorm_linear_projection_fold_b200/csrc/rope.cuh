// rope.cuh — rotary positions on heads that are already in memory, and (cos, sin) tables scaled for long
// contexts. The post-norm epilogue rotates whole heads in adjacent pairs while it has them in registers; these
// kernels serve everything else: projections without a per-head norm, the half layout, a rotated part of the
// head, and the gradient.
//
// A feature pair (a, b) of a row at position p turns by the angle of table row p:
//     a' = a c - b s,   b' = a s + b c        (RoFormer's rotation; the gradient is the transpose, s -> -s)
// Pairs are (2i, 2i+1) in the interleaved layout and (i, i + rot_dim / 2) in the half layout, i < rot_dim / 2;
// features from rot_dim on, and heads from n_rope_heads on, are carried over unchanged.
#pragma once

#include "sm100.cuh"

namespace fn {

struct RopeParams {
  const void* x;
  void* y;
  const float* cs;       // fp32 [max_pos][rot / 2][2]
  const int* positions;  // int32 [M]
  long long xs_row, xs_head, ys_row, ys_head;  // strides, elements
  long long items;       // threads with work: M * head_sets * units
  int H, hd, rot, n_rope, max_pos;
  int head_sets;  // a thread serves heads hs, hs + head_sets, ...
  int units;      // work units per head
  int in_place;   // y is x: what is not rotated is left where it is
  float sign;     // +1, or -1 for the gradient
};

// VEC consecutive features of type T, 2 to 16 bytes, as they lie in memory.
template <typename T, int VEC>
struct RopeVec {
  static constexpr int kBytes = VEC * static_cast<int>(sizeof(T));
  uint4 w;
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes == 16) {
      w = __ldcg(reinterpret_cast<const uint4*>(p));
    } else if constexpr (kBytes == 8) {
      const uint2 v = __ldcg(reinterpret_cast<const uint2*>(p));
      w.x = v.x, w.y = v.y;
    } else if constexpr (kBytes == 4) {
      w.x = __ldcg(reinterpret_cast<const uint32_t*>(p));
    } else {
      w.x = __ldcg(reinterpret_cast<const uint16_t*>(p));
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes == 16)
      *reinterpret_cast<uint4*>(p) = w;
    else if constexpr (kBytes == 8)
      *reinterpret_cast<uint2*>(p) = make_uint2(w.x, w.y);
    else if constexpr (kBytes == 4)
      *reinterpret_cast<uint32_t*>(p) = w.x;
    else
      *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w.x);
  }
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      f[e] = sizeof(T) == 4 ? __uint_as_float(v[e & 3]) : e & 1 ? bf16hi_to_f32(v[e >> 1]) : bf16lo_to_f32(v[e >> 1]);
  }
  __device__ __forceinline__ void set(const float (&f)[VEC]) {
    uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if constexpr (sizeof(T) == 4)
        v[e] = __float_as_uint(f[e]);
      else if (VEC == 1)
        v[0] = pack_bf16x2(f[0], 0.f);
      else if (e & 1)
        v[e >> 1] = pack_bf16x2(f[e & ~1], f[e]);
    }
    w = make_uint4(v[0], v[1], v[2], v[3]);
  }
};

// T: uint16_t (bf16) or float. VEC: features per access, a power of two of up to 16 bytes, as alignment and sizes allow.
// HALF layout: unit u < rot/2/VEC turns the VEC pairs from feature u VEC and their partners; later units carry VEC
// features over. Interleaved: with VEC > 1 unit u holds features u VEC .. (whole pairs, each turned or carried
// over); with VEC == 1 unit u < rot/2 is one pair and later units single features.
//
// Bound: HBM (each feature read and written once). A (cos, sin) pair is twice to four times as many bytes as the
// feature it turns, so a thread keeps the pairs of its unit in registers and serves several heads with them. All heads of a
// batch are loaded before any is stored (128 bytes in flight per thread): x and y may be the same memory, so the compiler
// cannot reorder them itself. x is read once, past the L1; positions and table by
// many threads of an SM, with plain (coherent) loads through it (positions past the L1: 71 us): the kernel before may have written
// any of them. 8192 x 96 x 128 bf16: 403 MB in 68 us (83 with one load in flight); 8192 x 48 heads of
// 108 features, 72 rotated, in accesses of four: 37 us (77 feature by feature).
template <typename T, int VEC, bool HALF>
__global__ void __launch_bounds__(256) k_rope(RopeParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= p.items) return;
  const int per_row = p.head_sets * p.units;
  const long long m = p.items <= 0xffffffffll ? static_cast<uint32_t>(id) / static_cast<uint32_t>(per_row) : id / per_row;
  const uint32_t in_row = static_cast<uint32_t>(id - m * per_row);
  const int hs = static_cast<int>(in_row / static_cast<uint32_t>(p.units)), u = static_cast<int>(in_row) - hs * p.units;
  constexpr bool kPairUnits = HALF || VEC == 1;          // a rotated unit is VEC features and their partners
  constexpr int NP = kPairUnits ? VEC : VEC / 2;          // pairs of a unit
  constexpr int kBatch = kPairUnits ? 4 : 8;              // heads in flight
  const int half = p.rot >> 1;
  const int rot_units = kPairUnits ? half / VEC : (p.rot + VEC - 1) / VEC;
  const bool turned = u < rot_units;
  // first feature of the unit, and (pair units) of its partners
  int f0, f1 = 0;
  if (HALF) {
    f0 = turned ? u * VEC : p.rot + (u - rot_units) * VEC;
    f1 = half + u * VEC;
  } else if (VEC == 1) {
    f0 = turned ? 2 * u : p.rot + (u - rot_units);
    f1 = f0 + 1;
  } else {
    f0 = u * VEC;
  }
  const T* x = static_cast<const T*>(p.x) + m * p.xs_row;
  T* y = static_cast<T*>(p.y) + m * p.ys_row;
  RopeVec<T, VEC> a[kBatch], b[kPairUnits ? kBatch : 1];
  // heads that are only carried over stay where they are in place
  auto has_work = [&](int h) { return h < p.H && !(p.in_place && !(turned && h < p.n_rope)); };
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * p.head_sets;
      if (!has_work(h)) continue;
      a[i].load(x + h * p.xs_head + f0);
      if (kPairUnits && turned) b[kPairUnits ? i : 0].load(x + h * p.xs_head + f1);
    }
  };
  load(hs);
  float c[NP], s[NP];
  if (turned && hs < p.n_rope) {
    const int pos = p.positions[m];
    if (static_cast<unsigned>(pos) < static_cast<unsigned>(p.max_pos)) {
      const int i0 = HALF ? u * VEC : f0 >> 1;  // first pair of the unit
      const float2* row = reinterpret_cast<const float2*>(p.cs) + static_cast<size_t>(pos) * half;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        // a unit that straddles rot_dim (interleaved): its last pairs are carried over and have no table entry
        const float2 v = i0 + j < half ? row[i0 + j] : make_float2(1.f, 0.f);
        c[j] = v.x;
        s[j] = p.sign * v.y;
      }
    } else {  // the row's rotated features become NaN; the host learns of it from the status word
#pragma unroll
      for (int j = 0; j < NP; ++j) c[j] = s[j] = __int_as_float(0x7fc00000);
      atomicOr(&g_device_status, kStatusBadPosition);
    }
  }
  for (int h0 = hs; h0 < p.H; h0 += kBatch * p.head_sets) {
    if (h0 != hs) load(h0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * p.head_sets;
      if (!has_work(h)) continue;
      T* yh = y + h * p.ys_head;
      if (turned && h < p.n_rope) {
        float v[VEC];
        a[i].get(v);
        if constexpr (kPairUnits) {
          float w[VEC];
          b[i].get(w);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float t0 = v[j], t1 = w[j];
            v[j] = t0 * c[j] - t1 * s[j];
            w[j] = t0 * s[j] + t1 * c[j];
          }
          b[i].set(w);
        } else {
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            const float t0 = v[2 * j], t1 = v[2 * j + 1];
            if (f0 + 2 * j < p.rot) {
              v[2 * j] = t0 * c[j] - t1 * s[j];
              v[2 * j + 1] = t0 * s[j] + t1 * c[j];
            }
          }
        }
        // a pair past rot_dim keeps its bits: conversions there and back are exact, NaN payloads aside, so only whole
        // units without such pairs go through them unconditionally
        if constexpr (!kPairUnits && sizeof(T) == 2) {
          const uint4 old = a[i].w;
          a[i].set(v);
          if (f0 + 2 >= p.rot) a[i].w.y = old.y;
          if (f0 + 4 >= p.rot) a[i].w.z = old.z;
          if (f0 + 6 >= p.rot) a[i].w.w = old.w;
        } else {
          a[i].set(v);
        }
      }
      a[i].store(yh + f0);
      if (kPairUnits && turned) b[kPairUnits ? i : 0].store(yh + f1);
    }
  }
}

// Scaled table. theta_i = base^(-2i/D) (D = rot_dim), then
//   linear  theta_i / factor (position interpolation)
//   ntk     base -> base factor^(D/(D-2)): the fastest pair keeps its angle, the slowest is divided by factor
//   yarn    by parts: a pair that turns t_i = original theta_i / 2 pi times within the original context keeps
//           theta_i for t_i >= beta, takes theta_i / factor for t_i <= alpha, and a linear blend between
//           ("YaRN: Efficient Context Window Extension of Large Language Models", NTK-by-parts)
// and both cos and sin are multiplied by `mscale`.
struct RopeTableParams {
  float* cs;
  int max_pos, half;
  int kind;  // 0 none, 1 linear, 2 ntk, 3 yarn
  double log2_base;  // ntk's factor included
  double factor, original, alpha, beta, mscale;
};

// A block holds 32 pairs (one per lane) and kRopeTableBlock positions p0 + 32 k + j. An entry is the product of
// exp(i theta j), in the registers of warp j % 8, and exp(i theta (p0 + 32 k)), in shared memory: two products and two
// fused multiply-adds in double precision, whose error, a few 2^-53, is far under the fp32 rounding at the end. Each
// thread starts from two sincospi and reaches the other factors by multiplication, with the warps' help. Angles are taken in
// half turns, so that reducing a large one is exact. Bound: the writes (131072 x 64 pairs: 67 MB in 14.6 us; with the entries
// made up, 13.4).
constexpr int kRopeTableFine = 32, kRopeTableCoarse = 16, kRopeTableBlock = kRopeTableFine * kRopeTableCoarse;

__device__ __forceinline__ double2 cmul(double2 a, double2 b) {
  return make_double2(a.x * b.x - a.y * b.y, a.x * b.y + a.y * b.x);
}
__device__ __forceinline__ double2 turn_pi(double half_turns) {
  double2 r;
  sincospi(half_turns, &r.y, &r.x);
  return r;
}

__global__ void __launch_bounds__(256) k_rope_table_scaled(RopeTableParams p) {
  __shared__ double2 fine[8][32], coarse[kRopeTableCoarse][32];
  static_assert(kRopeTableCoarse == 16, "two per warp");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.y * 32 + lane;
  const long long p0 = static_cast<long long>(blockIdx.x) * kRopeTableBlock;
  const int positions = static_cast<int>(min(static_cast<long long>(kRopeTableBlock), p.max_pos - p0));
  double theta = exp2(-p.log2_base * (static_cast<double>(i) / p.half));
  if (p.kind == 1) theta /= p.factor;
  if (p.kind == 3) {
    const double turns = p.original * theta / 6.283185307179586476925;
    const double keep = fmin(fmax((turns - p.alpha) / (p.beta - p.alpha), 0.0), 1.0);
    theta *= keep + (1.0 - keep) / p.factor;
  }
  const double t = theta / 3.14159265358979323846;
  double2 f[kRopeTableFine / 8];
  f[0] = turn_pi(warp * t);
  const double2 c0 = turn_pi(static_cast<double>(p0 + kRopeTableFine * warp) * t);
  fine[warp][lane] = f[0];
  coarse[warp][lane] = c0;
  __syncthreads();
  {
    const double2 step = cmul(fine[7][lane], fine[1][lane]);  // 8 positions
    const double2 back = make_double2(coarse[0][lane].x, -coarse[0][lane].y);
    // 8 x 32 positions: from p0 to p0 + 32, and to p0 + 7 x 32
    const double2 cstep = cmul(cmul(coarse[1][lane], back), cmul(coarse[7][lane], back));
    coarse[warp + 8][lane] = cmul(c0, cstep);
    f[0].x *= p.mscale;
    f[0].y *= p.mscale;
#pragma unroll
    for (int j = 1; j < kRopeTableFine / 8; ++j) f[j] = cmul(f[j - 1], step);
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  if (i >= p.half) return;
  float2* out = reinterpret_cast<float2*>(p.cs) + static_cast<size_t>(p0) * p.half + i;
#pragma unroll 2
  for (int k = 0; k * kRopeTableFine < positions; ++k) {
    const double2 b = coarse[k][lane];
#pragma unroll
    for (int j = 0; j < kRopeTableFine / 8; ++j) {
      const int pos = k * kRopeTableFine + warp + 8 * j;
      const double2 v = cmul(f[j], b);
      if (pos < positions) out[static_cast<size_t>(pos) * p.half] = make_float2(static_cast<float>(v.x), static_cast<float>(v.y));
    }
  }
}

}  // namespace fn
