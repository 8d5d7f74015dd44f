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

// One element of VEC consecutive features of type T, as floats.
template <typename T, int VEC>
struct RopeVec {
  float f[VEC];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 1) {
      if constexpr (sizeof(T) == 2)
        f[0] = __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << 16);
      else
        f[0] = *reinterpret_cast<const float*>(p);
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2) {
          f[2 * e] = bf16lo_to_f32(w[e]);
          f[2 * e + 1] = bf16hi_to_f32(w[e]);
        } else {
          f[e] = __uint_as_float(w[e]);
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC == 1) {
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(pack_bf16x2(f[0], 0.f) & 0xFFFFu);
      else
        *reinterpret_cast<float*>(p) = f[0];
    } else {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2)
          w[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
        else
          w[e] = __float_as_uint(f[e]);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

// T: uint16_t (bf16) or float. VEC: features per access, 16 bytes' worth, or 1 where alignment or sizes forbid.
// HALF layout: unit u < rot/2/VEC turns the VEC pairs from feature u VEC and their partners; later units carry VEC
// features over. Interleaved: with VEC > 1 unit u holds features u VEC .. (whole pairs, each turned or carried
// over); with VEC == 1 unit u < rot/2 is one pair and later units single features.
//
// Bound: HBM (each feature read and written once). A (cos, sin) pair is twice to four times as many bytes as the
// feature it turns, so a thread keeps the pairs of its unit in registers and serves several heads with them.
template <typename T, int VEC, bool HALF>
__global__ void __launch_bounds__(256) k_rope(RopeParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= p.items) return;
  const int per_row = p.head_sets * p.units;
  const long long m = id / per_row;
  const int in_row = static_cast<int>(id - m * per_row);
  const int hs = in_row / p.units, u = in_row - hs * p.units;
  constexpr bool kPairUnits = HALF || VEC == 1;          // a rotated unit is VEC features and their partners
  constexpr int NP = kPairUnits ? VEC : VEC / 2;          // pairs of a unit
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
  float c[NP], s[NP];
  if (turned && hs < p.n_rope) {
    const int pos = p.positions[m];
    if (static_cast<unsigned>(pos) < static_cast<unsigned>(p.max_pos)) {
      const int i0 = HALF ? u * VEC : f0 >> 1;  // first pair of the unit
      const float2* row = reinterpret_cast<const float2*>(p.cs) + static_cast<size_t>(pos) * half;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        // a unit that straddles rot_dim (interleaved): its last pairs are carried over and have no table entry
        const float2 v = i0 + j < half ? __ldg(row + i0 + j) : make_float2(1.f, 0.f);
        c[j] = v.x;
        s[j] = p.sign * v.y;
      }
    } else {  // the row's rotated features become NaN; the host learns of it from the status word
#pragma unroll
      for (int j = 0; j < NP; ++j) c[j] = s[j] = __int_as_float(0x7fc00000);
      atomicOr(&g_device_status, kStatusBadPosition);
    }
  }
  const T* x = static_cast<const T*>(p.x) + m * p.xs_row;
  T* y = static_cast<T*>(p.y) + m * p.ys_row;
#pragma unroll 4
  for (int h = hs; h < p.H; h += p.head_sets) {
    const T* xh = x + h * p.xs_head;
    T* yh = y + h * p.ys_head;
    const bool rot = turned && h < p.n_rope;
    if (!rot) {
      if (p.in_place) continue;
      RopeVec<T, VEC> a;
      a.load(xh + f0);
      a.store(yh + f0);
      if (kPairUnits && turned) {
        a.load(xh + f1);
        a.store(yh + f1);
      }
      continue;
    }
    RopeVec<T, VEC> a;
    a.load(xh + f0);
    if constexpr (kPairUnits) {
      RopeVec<T, VEC> b;
      b.load(xh + f1);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float t0 = a.f[j], t1 = b.f[j];
        a.f[j] = t0 * c[j] - t1 * s[j];
        b.f[j] = t0 * s[j] + t1 * c[j];
      }
      a.store(yh + f0);
      b.store(yh + f1);
    } else {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const float t0 = a.f[2 * j], t1 = a.f[2 * j + 1];
        if (f0 + 2 * j < p.rot) {
          a.f[2 * j] = t0 * c[j] - t1 * s[j];
          a.f[2 * j + 1] = t0 * s[j] + t1 * c[j];
        }
      }
      a.store(yh + f0);
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
  long long pstep;  // threads of one pair, and the distance between a thread's positions
  int kind;  // 0 none, 1 linear, 2 ntk, 3 yarn
  double base, factor, original, alpha, beta, mscale;
};

constexpr int kRopeTablePos = 64;  // positions of one thread, at most

// A thread owns one pair and up to kRopeTablePos positions `pstep` apart. It takes the angle of its first position and
// the step's angle in double precision, and reaches the others by complex multiplication in double precision (four
// products each; 63 steps cost about 63 * 2^-52, far under the fp32 rounding at the end). Bound: HBM writes; one
// fp64 sincos per entry instead is bound by the fp64 pipe.
__global__ void __launch_bounds__(256) k_rope_table_scaled(RopeTableParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const int i = static_cast<int>(id % p.half);
  const long long slot = id / p.half;  // threads of one pair: slots 0 .. pstep-1 start at position = slot
  const long long pstep = p.pstep;
  if (slot >= pstep) return;
  const double D = 2.0 * p.half;
  const double base = p.kind == 2 ? p.base * pow(p.factor, D / (D - 2.0)) : p.base;
  double theta = pow(base, -2.0 * i / D);
  if (p.kind == 1) theta /= p.factor;
  if (p.kind == 3) {
    const double turns = p.original * theta / 6.283185307179586476925;
    const double keep = fmin(fmax((turns - p.alpha) / (p.beta - p.alpha), 0.0), 1.0);
    theta *= keep + (1.0 - keep) / p.factor;
  }
  double c, s, dc, ds;
  sincos(static_cast<double>(slot) * theta, &s, &c);
  sincos(static_cast<double>(pstep) * theta, &ds, &dc);
  c *= p.mscale;
  s *= p.mscale;
  float2* out = reinterpret_cast<float2*>(p.cs) + i;
  for (long long pos = slot; pos < p.max_pos; pos += pstep) {
    out[pos * p.half] = make_float2(static_cast<float>(c), static_cast<float>(s));
    const double nc = c * dc - s * ds;
    s = c * ds + s * dc;
    c = nc;
  }
}

}  // namespace fn
