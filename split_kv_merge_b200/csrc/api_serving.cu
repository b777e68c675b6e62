// C ABI of the serving operators around the attention calls: rotary positions and the cache
// append.  Argument checks only; the work is in rope.cu and kv_append.cu.
#include <cuda_runtime.h>

#include <cmath>

#include "rope.cuh"

using namespace skv;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
skv_status cuda_status(int e) { return e == 0 ? SKV_OK : SKV_ERR_CUDA; }

skv_status check_rope(const skv_rope& r, int32_t head_dim) {
  if (r.dim < 0 || r.dim > head_dim) return SKV_ERR_INVALID;
  if (r.dim % 16 != 0 || r.dim > rope::kMaxDim) return SKV_ERR_UNSUPPORTED;
  if (r.dim == 0) return SKV_OK;
  if (r.layout != SKV_ROPE_INTERLEAVED && r.layout != SKV_ROPE_HALVES) return SKV_ERR_INVALID;
  if (!(r.mscale > 0.f) || !std::isfinite(r.mscale)) return SKV_ERR_INVALID;
  if (r.inv_freq_h == nullptr) {
    if (!(r.theta >= 1.0) || !std::isfinite(r.theta)) return SKV_ERR_INVALID;
  } else {
    for (int32_t i = 0; i < r.dim / 2; ++i)
      if (!(std::fabs(r.inv_freq_h[i]) < 4294967296.0)) return SKV_ERR_INVALID;  // also NaN
  }
  return SKV_OK;
}

// Strides of a [rows, heads, dim] tensor whose element is `size` bytes: multiples of 16 bytes.
skv_status check_rows(const void* base, const int64_t* stride, int64_t size) {
  if (base == nullptr || stride[0] < 0 || stride[1] < 0) return SKV_ERR_INVALID;
  if (!aligned16(base) || stride[0] * size % 16 != 0 || stride[1] * size % 16 != 0) return SKV_ERR_ALIGNMENT;
  return SKV_OK;
}

// Output rows, which may also be the input with the same strides.
skv_status check_out_rows(const void* out, const int64_t* out_stride, const void* in, const int64_t* in_stride,
                          int64_t size) {
  const skv_status st = check_rows(out, out_stride, size);
  if (st != SKV_OK) return st;
  if (out == in && (out_stride[0] != in_stride[0] || out_stride[1] != in_stride[1])) return SKV_ERR_INVALID;
  return SKV_OK;
}

}  // namespace

extern "C" {

skv_status skv_rope_frequencies(int32_t dim, double theta, int32_t scaling, double factor, double original_context,
                                double low, double high, double* inv_freq_h, float* mscale) {
  if (dim < 2 || dim % 2 != 0 || !(theta > 1.0) || !std::isfinite(theta)) return SKV_ERR_INVALID;
  if (scaling < SKV_ROPE_SCALE_NONE || scaling > SKV_ROPE_SCALE_BANDS) return SKV_ERR_INVALID;
  const bool ramp = scaling == SKV_ROPE_SCALE_YARN || scaling == SKV_ROPE_SCALE_BANDS;
  if (scaling != SKV_ROPE_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return SKV_ERR_INVALID;
  if (scaling == SKV_ROPE_SCALE_NTK && dim <= 2) return SKV_ERR_INVALID;
  if (ramp && (!(original_context > 0.0) || !std::isfinite(original_context) || !(low > 0.0) || !(high > low) ||
               !std::isfinite(high)))
    return SKV_ERR_INVALID;
  const double two_pi = 6.283185307179586476925286766559;
  const int32_t half = dim / 2;
  const double base = scaling == SKV_ROPE_SCALE_NTK ? theta * std::pow(factor, (double)dim / (dim - 2)) : theta;
  // pair index at which a frequency turns `n` times over the original context
  auto pair_at = [&](double n) { return dim * std::log(original_context / (n * two_pi)) / (2.0 * std::log(theta)); };
  double first = 0, last = 0;
  if (scaling == SKV_ROPE_SCALE_YARN) {
    first = std::fmax(std::floor(pair_at(high)), 0.0);
    last = std::fmin(std::ceil(pair_at(low)), (double)dim - 1);
    if (last <= first) last = first + 0.001;
  }
  for (int32_t i = 0; i < half && inv_freq_h != nullptr; ++i) {
    double f = std::pow(base, -2.0 * i / dim);
    if (scaling == SKV_ROPE_SCALE_LINEAR) {
      f /= factor;
    } else if (scaling == SKV_ROPE_SCALE_YARN) {
      const double stretched = std::fmin(1.0, std::fmax(0.0, (i - first) / (last - first)));
      f = f / factor * stretched + f * (1.0 - stretched);
    } else if (scaling == SKV_ROPE_SCALE_BANDS) {
      const double turns = original_context * f / two_pi;
      const double kept = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
      f = f / factor * (1.0 - kept) + f * kept;
    }
    inv_freq_h[i] = f;
  }
  if (mscale != nullptr) *mscale = scaling == SKV_ROPE_SCALE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return SKV_OK;
}

skv_status skv_rope_apply(const skv_rope_params* p, skv_stream_t stream) {
  if (p == nullptr || p->num_tokens < 0 || p->num_q_heads < 0 || p->num_k_heads < 0) return SKV_ERR_INVALID;
  if (p->head_dim < 1) return SKV_ERR_INVALID;
  if (p->head_dim % 8 != 0 || p->head_dim > 1024) return SKV_ERR_UNSUPPORTED;
  if (p->dtype != SKV_BF16 && p->dtype != SKV_F32) return SKV_ERR_UNSUPPORTED;
  skv_status st = check_rope(p->rope, p->head_dim);
  if (st != SKV_OK) return st;
  if (p->num_tokens == 0 || (p->num_q_heads == 0 && p->num_k_heads == 0)) return SKV_OK;
  if ((int64_t)p->num_q_heads + p->num_k_heads > 65535) return SKV_ERR_UNSUPPORTED;
  const int64_t size = p->dtype == SKV_F32 ? 4 : 2;
  if (p->num_q_heads > 0) {
    st = check_rows(p->q, p->q_stride, size);
    if (st == SKV_OK) st = check_out_rows(p->q_out, p->q_out_stride, p->q, p->q_stride, size);
    if (st != SKV_OK) return st;
  }
  if (p->num_k_heads > 0) {
    st = check_rows(p->k, p->k_stride, size);
    if (st == SKV_OK) st = check_out_rows(p->k_out, p->k_out_stride, p->k, p->k_stride, size);
    if (st != SKV_OK) return st;
  }
  if (p->rope.dim > 0 && p->positions == nullptr) return SKV_ERR_INVALID;
  return cuda_status(launch_rope(*p, reinterpret_cast<cudaStream_t>(stream)));
}

skv_status skv_paged_kv_append(const skv_append_params* p, skv_stream_t stream) {
  if (p == nullptr || p->batch < 0 || p->num_rows < 0 || p->num_pages < 0 || p->page_size < 1) return SKV_ERR_INVALID;
  if (p->num_kv_heads < 1 || p->num_q_heads < 0) return SKV_ERR_INVALID;
  if (p->head_dim != 64 && p->head_dim != 128) return SKV_ERR_UNSUPPORTED;
  if ((int64_t)2 * p->num_kv_heads + p->num_q_heads > 65535) return SKV_ERR_UNSUPPORTED;
  if (p->kv_dtype != SKV_BF16 && p->kv_dtype != SKV_E4M3 && p->kv_dtype != SKV_I8) return SKV_ERR_UNSUPPORTED;
  skv_status st = check_rope(p->rope, p->head_dim);
  if (st != SKV_OK) return st;
  const bool scaled = p->block_tokens != 0;
  if (p->block_tokens < 0) return SKV_ERR_INVALID;
  if (scaled) {
    if (p->kv_dtype == SKV_BF16) return SKV_ERR_INVALID;
    if (p->block_tokens > 256) return SKV_ERR_UNSUPPORTED;
    if (p->page_size % p->block_tokens != 0) return SKV_ERR_INVALID;
  } else if (p->kv_dtype == SKV_I8) {
    return SKV_ERR_UNSUPPORTED;
  } else if (p->kv_dtype == SKV_E4M3 && !(p->kv_scale > 0.f && std::isfinite(p->kv_scale) && std::isfinite(1.f / p->kv_scale))) {
    return SKV_ERR_INVALID;
  }
  if (p->num_rows == 0 || p->batch == 0) return SKV_OK;
  if (!p->append_indptr || !p->kv_indptr || !p->kv_indices || !p->kv_last_page_len) return SKV_ERR_INVALID;
  if (!p->k_cache || !p->v_cache || (scaled && (!p->k_scale || !p->v_scale))) return SKV_ERR_INVALID;
  st = check_rows(p->k, p->k_row_stride, 2);
  if (st == SKV_OK) st = check_rows(p->v, p->v_row_stride, 2);
  if (st != SKV_OK) return st;
  const int64_t size = p->kv_dtype == SKV_BF16 ? 2 : 1;
  for (int i = 0; i < 3; ++i) {
    if (p->k_stride[i] < 0 || p->v_stride[i] < 0) return SKV_ERR_INVALID;
    if (p->k_stride[i] * size % 16 != 0 || p->v_stride[i] * size % 16 != 0) return SKV_ERR_ALIGNMENT;
    if (scaled && (p->k_scale_stride[i] < 0 || p->v_scale_stride[i] < 0)) return SKV_ERR_INVALID;
  }
  if (!aligned16(p->k_cache) || !aligned16(p->v_cache)) return SKV_ERR_ALIGNMENT;
  if (p->num_q_heads > 0) {
    st = check_rows(p->q, p->q_stride, 2);
    if (st == SKV_OK) st = check_out_rows(p->q_out, p->q_out_stride, p->q, p->q_stride, 2);
    if (st != SKV_OK) return st;
  }
  return cuda_status(launch_kv_append(*p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
