// api_rope.cuh — host side of rope.cuh: checks, the choice of access width and the launches. Part of flashnorm.cu.
#pragma once

namespace {

// Heads per thread: a thread's (cos, sin) pairs serve this many heads (fewer while there are too few threads to
// fill the device).
int rope_head_sets(int64_t M, int64_t H, int64_t units, int sms) {
  const int64_t enough = static_cast<int64_t>(sms) * 2048;  // one thread per resident slot
  int64_t per = 8;
  while (per > 1 && M * ((H + per - 1) / per) * units < enough) per >>= 1;
  return static_cast<int>((H + per - 1) / per);
}

template <typename T, int VEC, bool HALF>
fn_status launch_rope(const fn::RopeParams& p, cudaStream_t s) {
  const long long blocks = (p.items + 255) / 256;
  if (blocks > kMaxDim) return fail(FN_ERR_UNSUPPORTED, "too many heads for one launch");
  cudaError_t e = launch_kernel(fn::k_rope<T, VEC, HALF>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, 1, p);
  if (e != cudaSuccess) return cuda_fail(e, "rope launch");
  return FN_OK;
}

}  // namespace

extern "C" {

fn_status flashnorm_rope(const void* x, const void* rope_cs, const void* positions, void* y, int64_t M, int64_t H,
                         int64_t head_dim, int64_t rot_dim, int64_t n_rope_heads, int64_t max_pos,
                         int64_t x_row_stride, int64_t x_head_stride, int64_t y_row_stride, int64_t y_head_stride,
                         int layout, int backward, int dtype, void* stream) {
  g_last_error[0] = '\0';
  if (M < 0 || M > kMaxDim) return fail(FN_ERR_INVALID_ARG, "M = %lld out of range", (long long)M);
  if (H < 1 || H > 65536) return fail(FN_ERR_INVALID_ARG, "H = %lld must be in [1, 65536]", (long long)H);
  if (head_dim < 2 || head_dim > 65536) return fail(FN_ERR_INVALID_ARG, "head_dim = %lld must be in [2, 65536]", (long long)head_dim);
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > head_dim)
    return fail(FN_ERR_INVALID_ARG, "rot_dim = %lld must be even and in [2, head_dim]", (long long)rot_dim);
  if (n_rope_heads < 0 || n_rope_heads > H) return fail(FN_ERR_INVALID_ARG, "n_rope_heads = %lld out of range", (long long)n_rope_heads);
  if (max_pos < 1 || max_pos > kMaxDim) return fail(FN_ERR_INVALID_ARG, "max_pos = %lld out of range", (long long)max_pos);
  if (layout != FN_ROPE_INTERLEAVED && layout != FN_ROPE_HALF) return fail(FN_ERR_INVALID_ARG, "layout %d unknown", layout);
  if (backward != 0 && backward != 1) return fail(FN_ERR_INVALID_ARG, "backward must be 0 or 1");
  if (dtype != FN_BF16 && dtype != FN_F32) return fail(FN_ERR_INVALID_ARG, "dtype %d unknown", dtype);
  if (H * head_dim > kMaxDim) return fail(FN_ERR_UNSUPPORTED, "rows of %lld features", (long long)(H * head_dim));
  if (x_head_stride < 0 || x_row_stride < 0 || x_head_stride > (int64_t{1} << 40) || x_row_stride > (int64_t{1} << 40) ||
      y_head_stride > (int64_t{1} << 40) || y_row_stride > (int64_t{1} << 40))
    return fail(FN_ERR_INVALID_ARG, "stride out of range");
  // y holds every feature in a place of its own: rows of heads, or heads of rows
  const bool rows_of_heads = (H == 1 || y_head_stride >= head_dim) &&
                             (M <= 1 || y_row_stride >= (H - 1) * y_head_stride + head_dim);
  const bool heads_of_rows = (M <= 1 || y_row_stride >= head_dim) &&
                             (H == 1 || (y_head_stride >= head_dim &&
                                         (M <= 1 || (y_head_stride - head_dim) / y_row_stride >= M - 1)));
  if (y_row_stride < 0 || y_head_stride < 0 || (!rows_of_heads && !heads_of_rows))
    return fail(FN_ERR_INVALID_ARG, "the rows and heads of y overlap");
  const bool in_place = x == y && M > 0;  // empty tensors all have the address 0
  if (in_place && (x_row_stride != y_row_stride || x_head_stride != y_head_stride))
    return fail(FN_ERR_INVALID_ARG, "in place, x and y must have the same strides");
  if (M == 0) return FN_OK;
  const uintptr_t es = dtype == FN_BF16 ? 2 : 4;
  if (x == nullptr || y == nullptr) return fail(FN_ERR_INVALID_ARG, "x or y is NULL");
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) % es)
    return fail(FN_ERR_ALIGN, "x or y is not aligned to its elements");
  fn_status st;
  if ((st = check_ptr(rope_cs, "rope_cs")) != FN_OK) return st;
  if (positions == nullptr) return fail(FN_ERR_INVALID_ARG, "positions is NULL");
  if (reinterpret_cast<uintptr_t>(positions) & 3u) return fail(FN_ERR_ALIGN, "positions is not 4-byte aligned");
  int dev = 0;
  const int sms = device_sm_count(&dev);
  if (sms <= 0) return fail(FN_ERR_CUDA, "cannot query the current device");
  // the widest access that bases, strides and sizes allow: 16 bytes, or less for heads like 38 or 210 features
  const bool half = layout == FN_ROPE_HALF;
  int v = static_cast<int>(16 / es);
  while (v > 1 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) % (v * es) != 0 ||
                   (head_dim | x_row_stride | x_head_stride | y_row_stride | y_head_stride | (half ? rot_dim / 2 : 0)) % v != 0))
    v /= 2;
  const int64_t units = half || v == 1 ? rot_dim / 2 / v + (head_dim - rot_dim) / v : head_dim / v;
  fn::RopeParams p;
  p.x = x;
  p.y = y;
  p.cs = static_cast<const float*>(rope_cs);
  p.positions = static_cast<const int*>(positions);
  p.xs_row = x_row_stride, p.xs_head = x_head_stride, p.ys_row = y_row_stride, p.ys_head = y_head_stride;
  p.H = static_cast<int>(H), p.hd = static_cast<int>(head_dim), p.rot = static_cast<int>(rot_dim);
  p.n_rope = static_cast<int>(n_rope_heads), p.max_pos = static_cast<int>(max_pos);
  p.units = static_cast<int>(units);
  p.head_sets = rope_head_sets(M, H, units, sms);
  p.items = M * p.head_sets * units;
  p.in_place = in_place ? 1 : 0;
  p.sign = backward ? -1.0f : 1.0f;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == FN_BF16) {
    switch (v) {
      case 8: return half ? launch_rope<uint16_t, 8, true>(p, s) : launch_rope<uint16_t, 8, false>(p, s);
      case 4: return half ? launch_rope<uint16_t, 4, true>(p, s) : launch_rope<uint16_t, 4, false>(p, s);
      case 2: return half ? launch_rope<uint16_t, 2, true>(p, s) : launch_rope<uint16_t, 2, false>(p, s);
      default: return half ? launch_rope<uint16_t, 1, true>(p, s) : launch_rope<uint16_t, 1, false>(p, s);
    }
  }
  switch (v) {
    case 4: return half ? launch_rope<float, 4, true>(p, s) : launch_rope<float, 4, false>(p, s);
    case 2: return half ? launch_rope<float, 2, true>(p, s) : launch_rope<float, 2, false>(p, s);
    default: return half ? launch_rope<float, 1, true>(p, s) : launch_rope<float, 1, false>(p, s);
  }
}

fn_status flashnorm_rope_table_scaled(void* rope_cs, int64_t max_pos, int64_t rot_dim, double base, int scaling,
                                      double factor, double original_max_pos, double alpha, double beta,
                                      double attention_factor, void* stream) {
  g_last_error[0] = '\0';
  if (max_pos < 1 || max_pos > kMaxDim) return fail(FN_ERR_INVALID_ARG, "max_pos = %lld out of range", (long long)max_pos);
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 65536)
    return fail(FN_ERR_INVALID_ARG, "rot_dim = %lld must be even and in [2, 65536]", (long long)rot_dim);
  if (!(base > 1.0) || !std::isfinite(base)) return fail(FN_ERR_INVALID_ARG, "base must be finite and > 1");
  if (scaling < FN_ROPE_SCALE_NONE || scaling > FN_ROPE_SCALE_YARN) return fail(FN_ERR_INVALID_ARG, "scaling %d unknown", scaling);
  if (scaling != FN_ROPE_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(FN_ERR_INVALID_ARG, "factor must be finite and >= 1");
  if (scaling == FN_ROPE_SCALE_NTK && rot_dim < 4) return fail(FN_ERR_INVALID_ARG, "ntk scaling needs rot_dim >= 4");
  if (scaling == FN_ROPE_SCALE_YARN &&
      (!(original_max_pos > 0.0) || !std::isfinite(original_max_pos) || !(alpha >= 0.0) || !(beta > alpha) || !std::isfinite(beta)))
    return fail(FN_ERR_INVALID_ARG, "yarn scaling needs original_max_pos > 0 and 0 <= alpha < beta");
  if (!(attention_factor > 0.0) || !std::isfinite(attention_factor))
    return fail(FN_ERR_INVALID_ARG, "attention_factor must be finite and > 0");
  fn_status st;
  if ((st = check_ptr(rope_cs, "rope_cs")) != FN_OK) return st;
  fn::RopeTableParams p;
  p.cs = static_cast<float*>(rope_cs);
  p.max_pos = static_cast<int>(max_pos);
  p.half = static_cast<int>(rot_dim / 2);
  p.kind = scaling;
  const long double D = static_cast<long double>(rot_dim);
  p.log2_base = static_cast<double>(std::log2(static_cast<long double>(base)) +
                                    (scaling == FN_ROPE_SCALE_NTK ? std::log2(static_cast<long double>(factor)) * D / (D - 2) : 0.0L));
  p.factor = factor, p.original = original_max_pos, p.alpha = alpha, p.beta = beta;
  p.mscale = attention_factor;
  const int64_t blocks = (max_pos + fn::kRopeTableBlock - 1) / fn::kRopeTableBlock;
  cudaError_t e = launch_kernel(fn::k_rope_table_scaled, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>((p.half + 31) / 32)),
                                dim3(256), 0, static_cast<cudaStream_t>(stream), 1, p);
  if (e != cudaSuccess) return cuda_fail(e, "scaled rope table launch");
  return FN_OK;
}

}  // extern "C"
