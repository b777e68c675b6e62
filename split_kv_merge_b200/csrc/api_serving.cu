// C ABI of the serving operators around the paged attention calls: rotary positions, the cache
// append and packed prompt attention.  Argument checks and the prompt planner; the work is in
// rope.cu, kv_append.cu and prompt_attn.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <queue>
#include <vector>

#include "prompt_plan.h"
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

// Whether the rows (`extent` values each) of a strided array lie apart: taken by size, every stride spans the
// dimensions before it.
template <int N>
bool rows_apart(const int64_t (&count)[N], const int64_t* stride, int64_t extent) {
  int64_t st[N], n[N];
  int dims = 0;
  for (int i = 0; i < N; ++i) {
    if (count[i] <= 1) continue;  // its stride is never used
    int at = dims++;
    for (; at > 0 && st[at - 1] > stride[i]; --at) st[at] = st[at - 1], n[at] = n[at - 1];
    st[at] = stride[i], n[at] = count[i];
  }
  __int128 span = extent;
  for (int i = 0; i < dims; ++i) {
    if (st[i] < span) return false;
    span += (__int128)st[i] * (n[i] - 1);
  }
  return true;
}

// Output rows, which may also be the input with the same strides; each has a place of its own.
skv_status check_out_rows(const void* out, const int64_t* out_stride, const void* in, const int64_t* in_stride,
                          int64_t size, int64_t tokens, int64_t heads, int64_t head_dim) {
  const skv_status st = check_rows(out, out_stride, size);
  if (st != SKV_OK) return st;
  if (!rows_apart<2>({tokens, heads}, out_stride, head_dim)) return SKV_ERR_INVALID;
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
    if (st == SKV_OK)
      st = check_out_rows(p->q_out, p->q_out_stride, p->q, p->q_stride, size, p->num_tokens, p->num_q_heads,
                          p->head_dim);
    if (st != SKV_OK) return st;
  }
  if (p->num_k_heads > 0) {
    st = check_rows(p->k, p->k_stride, size);
    if (st == SKV_OK)
      st = check_out_rows(p->k_out, p->k_out_stride, p->k, p->k_stride, size, p->num_tokens, p->num_k_heads,
                          p->head_dim);
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
  } else if (p->kv_dtype == SKV_E4M3 &&
             !(p->kv_scale > 0.f && std::isfinite(p->kv_scale) && std::isfinite(1.f / p->kv_scale))) {
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
  // what is written has a place of its own
  const int64_t rows[3] = {p->num_pages, p->page_size, p->num_kv_heads};
  if (!rows_apart(rows, p->k_stride, p->head_dim) || !rows_apart(rows, p->v_stride, p->head_dim)) return SKV_ERR_INVALID;
  if (scaled) {
    const int64_t scales[3] = {p->num_pages, p->page_size / p->block_tokens, p->num_kv_heads};
    if (!rows_apart(scales, p->k_scale_stride, 1) || !rows_apart(scales, p->v_scale_stride, 1)) return SKV_ERR_INVALID;
  }
  if (!aligned16(p->k_cache) || !aligned16(p->v_cache)) return SKV_ERR_ALIGNMENT;
  if (p->num_q_heads > 0) {
    st = check_rows(p->q, p->q_stride, 2);
    if (st == SKV_OK)
      st = check_out_rows(p->q_out, p->q_out_stride, p->q, p->q_stride, 2, p->num_rows, p->num_q_heads, p->head_dim);
    if (st != SKV_OK) return st;
  }
  return cuda_status(launch_kv_append(*p, reinterpret_cast<cudaStream_t>(stream)));
}

skv_status skv_plan_prompt(int32_t batch, const int32_t* qo_indptr_h, const int32_t* kv_indptr_h,
                           int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim, int32_t causal,
                           int32_t num_sms, int32_t* plan_h, int64_t plan_capacity, skv_plan_info* info) try {
  if (info == nullptr) return SKV_ERR_INVALID;
  std::memset(info, 0, sizeof(*info));
  if (batch < 0 || qo_indptr_h == nullptr || num_qo_heads < 1 || num_kv_heads < 1) return SKV_ERR_INVALID;
  if (num_qo_heads % num_kv_heads != 0 || num_sms < 0) return SKV_ERR_INVALID;
  if (head_dim != 64 && head_dim != 128) return SKV_ERR_UNSUPPORTED;
  if (num_qo_heads > 65535) return SKV_ERR_UNSUPPORTED;
  const int32_t* kv = kv_indptr_h != nullptr ? kv_indptr_h : qo_indptr_h;
  if (qo_indptr_h[0] != 0 || kv[0] != 0) return SKV_ERR_INVALID;
  for (int32_t r = 0; r < batch; ++r)
    if (qo_indptr_h[r + 1] < qo_indptr_h[r] || kv[r + 1] < kv[r]) return SKV_ERR_INVALID;
  const int32_t ctas = num_sms > 0 ? num_sms : device_sm_count();
  const bool heads = (num_qo_heads / num_kv_heads) % 2 == 0;  // A and B: two heads, else two token tiles
  const int32_t step = heads ? kPromptTile : 2 * kPromptTile;

  // token tiles: first token, tokens, key tiles its last token needs
  struct Span {
    int32_t r, q0, n, tiles;
  };
  std::vector<Span> spans;
  int64_t total = 0;
  const int32_t head_items = heads ? num_qo_heads / 2 : num_qo_heads;
  for (int32_t r = 0; r < batch; ++r) {
    const int64_t n = (int64_t)qo_indptr_h[r + 1] - qo_indptr_h[r], len = (int64_t)kv[r + 1] - kv[r];
    for (int64_t q0 = 0; q0 < n; q0 += step) {
      const int64_t m = std::min<int64_t>(step, n - q0);
      const int64_t seen = causal ? std::min(len, std::max<int64_t>(0, len - n + q0 + m)) : len;
      const int64_t tiles = (seen + kPromptTile - 1) / kPromptTile;
      spans.push_back(Span{r, (int32_t)q0, (int32_t)m, (int32_t)tiles});
      total += std::max<int64_t>(tiles, 1) * head_items;
    }
  }
  // a span longer than 1.5 shares of the whole work is cut along the keys (pieces of >= 8 tiles)
  const int64_t chunk = std::max<int64_t>(8, (total + ctas - 1) / ctas);
  std::vector<int32_t> cuts(spans.size());
  bool whole = true;
  for (size_t i = 0; i < spans.size(); ++i) {
    cuts[i] = 2 * (int64_t)spans[i].tiles > 3 * chunk ? (int32_t)((spans[i].tiles + chunk - 1) / chunk) : 1;
    whole = whole && cuts[i] == 1;
  }
  // A few items per CTA leave some CTAs one item short.  Where that costs a twentieth, the spans of as many
  // of the shortest items as make no full round are cut too, if the longest CTA's share and the pass that
  // joins the partials (about 3 us and their bytes twice, at 1 us for half an item's tile) then end sooner.
  // 4096 query tokens over 16384 keys, 32/8 heads: 441 -> 395 tiles for the longest CTA.  Of 150 shapes (1 to 9
  // sequences of 300 .. 8000 query tokens over up to 16384 keys, 32/8, 16/2, 8/8, 12/4 and 64/8 heads, causal and
  // not) 31 are cut, each timed both ways: times of 0.69 to 1.00 of the whole items' for 29 of them, 0.91 in the
  // middle; 1.02 (2048 over 8048, 32/8) and 1.07 (2048 over 2048, 64/8, not causal) for the other two.
  const int64_t whole_items = (int64_t)spans.size() * head_items;
  if (whole && whole_items > ctas && whole_items < 8LL * ctas) {
    std::vector<int32_t> by_len(spans.size());
    for (size_t i = 0; i < by_len.size(); ++i) by_len[i] = (int32_t)i;
    std::stable_sort(by_len.begin(), by_len.end(),
                     [&](int32_t x, int32_t y) { return spans[x].tiles > spans[y].tiles; });
    const auto ends_at = [&](size_t cut, int32_t pieces) {  // the last `cut` of by_len in `pieces` each
      std::vector<int64_t> costs;
      costs.reserve((by_len.size() + cut * pieces) * head_items);
      int64_t rows = 0;
      for (size_t k = 0; k < by_len.size(); ++k) {
        const Span& s = spans[by_len[k]];
        const int32_t n = k + cut < by_len.size() ? 1 : pieces;
        if (n > 1) rows += (int64_t)s.n * n;
        for (int32_t j = 0; j < n; ++j) {
          const int64_t t = (int64_t)s.tiles * (j + 1) / n - (int64_t)s.tiles * j / n;
          costs.insert(costs.end(), head_items, t * (heads || s.n > kPromptTile ? 2 : 1) + 3);
        }
      }
      std::sort(costs.begin(), costs.end(), std::greater<int64_t>());
      std::priority_queue<int64_t, std::vector<int64_t>, std::greater<int64_t>> load;
      for (int32_t c = 0; c < ctas; ++c) load.push(0);
      int64_t most = 0;
      for (int64_t c : costs) {
        const int64_t l = load.top() + c;
        load.pop();
        load.push(l);
        most = std::max(most, l);
      }
      return most + (rows > 0 ? 3 + rows * num_qo_heads * head_dim * 8 / 6000000 : 0);
    };
    int64_t best = ends_at(0, 1), best_cut = 0, best_pieces = 1;
    if (best * 20 > 21 * (2 * total + 3 * whole_items) / ctas) {
      const int64_t cut = (whole_items % ctas + head_items - 1) / head_items;
      for (int32_t pieces : {2, 3, 4, 6}) {
        if (cut < 1 || spans[by_len.back()].tiles < 8 * pieces) break;
        const int64_t e = ends_at((size_t)cut, pieces);
        if (e < best) best = e, best_cut = cut, best_pieces = pieces;
      }
      for (int64_t k = 0; k < best_cut; ++k) cuts[by_len[by_len.size() - 1 - k]] = (int32_t)best_pieces;
    }
  }
  std::vector<PromptItem> items;
  std::vector<MergeItem> merges;
  int64_t part_rows = 0;
  for (size_t si = 0; si < spans.size(); ++si) {
    const Span& s = spans[si];
    const int64_t n = (int64_t)qo_indptr_h[s.r + 1] - qo_indptr_h[s.r], len = (int64_t)kv[s.r + 1] - kv[s.r];
    const int32_t pieces = cuts[si];
    info->max_splits = std::max(info->max_splits, pieces);
    info->total_splits += pieces;
    if (part_rows + (int64_t)s.n * pieces > INT32_MAX) return SKV_ERR_UNSUPPORTED;
    for (int32_t j = 0; j < pieces; ++j) {
      PromptItem w;
      std::memset(&w, 0, sizeof(w));
      w.q0a = qo_indptr_h[s.r] + s.q0;
      w.na = std::min(s.n, kPromptTile);
      w.limit_a = (int32_t)(len - n + s.q0 + 1);
      w.q0b = heads ? w.q0a : w.q0a + kPromptTile;
      w.nb = heads ? w.na : s.n - w.na;
      w.limit_b = heads ? w.limit_a : w.limit_a + kPromptTile;
      w.kv0 = kv[s.r];
      w.kv_len = (int32_t)len;
      w.tile_begin = (int32_t)((int64_t)s.tiles * j / pieces);
      w.tile_end = (int32_t)((int64_t)s.tiles * (j + 1) / pieces);
      w.part_row = pieces > 1 ? (int32_t)(part_rows + j) : -1;
      w.part_stride = pieces;
      w.causal = causal != 0;
      for (int32_t h = 0; h < num_qo_heads; h += heads ? 2 : 1) {
        w.ha = h;
        w.hb = heads ? h + 1 : h;
        items.push_back(w);
      }
    }
    if (pieces > 1) {
      for (int32_t t = 0; t < s.n; ++t)
        merges.push_back(MergeItem{qo_indptr_h[s.r] + s.q0 + t, (int32_t)(part_rows + (int64_t)t * pieces), pieces, 0});
      part_rows += (int64_t)s.n * pieces;
    }
  }
  // longest first onto the least loaded CTA; an item costs its tiles for both query tiles, and a
  // start and end worth about one and a half tiles
  const auto cost = [](const PromptItem& w) {
    return (int64_t)(w.tile_end - w.tile_begin) * (w.nb > 0 ? 2 : 1) + 3;
  };
  std::vector<int32_t> order(items.size());
  for (size_t i = 0; i < items.size(); ++i) order[i] = (int32_t)i;
  std::stable_sort(order.begin(), order.end(),
                   [&](int32_t x, int32_t y) { return cost(items[x]) > cost(items[y]); });
  const int32_t g = (int32_t)std::min<size_t>(items.size(), (size_t)ctas);
  using Load = std::pair<int64_t, int32_t>;
  std::priority_queue<Load, std::vector<Load>, std::greater<Load>> least;
  for (int32_t c = 0; c < g; ++c) least.push({0, c});
  std::vector<int32_t> owner(items.size()), indptr(g + 1, 0);
  for (int32_t i : order) {
    Load l = least.top();
    least.pop();
    owner[i] = l.second;
    ++indptr[l.second + 1];
    l.first += cost(items[i]);
    least.push(l);
  }
  for (int32_t c = 0; c < g; ++c) indptr[c + 1] += indptr[c];

  const int64_t words = 16LL * (int64_t)items.size() + 4LL * (int64_t)merges.size() + (g > 0 ? g + 1 : 0);
  if (words > INT32_MAX) return SKV_ERR_UNSUPPORTED;
  info->num_work = (int32_t)items.size();
  info->num_partial_rows = (int32_t)part_rows;
  info->num_merge_rows = (int32_t)merges.size();
  info->kernel = KERNEL_PROMPT;
  info->q_tile = kPromptTile;
  info->plan_words = (int32_t)words;
  info->num_ctas = g;
  info->cta_offset = (int32_t)(16LL * (int64_t)items.size() + 4LL * (int64_t)merges.size());
  if (plan_h == nullptr || plan_capacity < words) return words == 0 ? SKV_OK : SKV_ERR_WORKSPACE;
  std::vector<int32_t> at(indptr.begin(), indptr.end() - 1);
  PromptItem* out = reinterpret_cast<PromptItem*>(plan_h);
  for (int32_t i : order) out[at[owner[i]]++] = items[i];
  if (!merges.empty()) std::memcpy(plan_h + 16 * items.size(), merges.data(), merges.size() * sizeof(MergeItem));
  if (g > 0) std::memcpy(plan_h + info->cta_offset, indptr.data(), (g + 1) * sizeof(int32_t));
  return SKV_OK;
} catch (...) {
  return SKV_ERR_INVALID;  // out of host memory
}

skv_status skv_prompt_attn_fwd(const skv_prompt_params* p, const int32_t* plan_d, const skv_plan_info* info,
                               skv_stream_t stream) {
  if (p == nullptr || info == nullptr || info->kernel != KERNEL_PROMPT) return SKV_ERR_INVALID;
  if (info->num_work < 0 || info->num_merge_rows < 0 || info->num_partial_rows < 0) return SKV_ERR_INVALID;
  if (p->total_q < 0 || p->total_kv < 0 || p->num_qo_heads < 1 || p->num_kv_heads < 1) return SKV_ERR_INVALID;
  if (p->num_qo_heads % p->num_kv_heads != 0) return SKV_ERR_INVALID;
  if (p->head_dim != 64 && p->head_dim != 128) return SKV_ERR_UNSUPPORTED;
  if (p->num_qo_heads > 65535) return SKV_ERR_UNSUPPORTED;
  if (p->o_dtype != SKV_F32 && p->o_dtype != SKV_BF16) return SKV_ERR_UNSUPPORTED;
  if (!(p->sm_scale > 0.f) || !std::isfinite(p->sm_scale)) return SKV_ERR_INVALID;
  if (info->num_work == 0 || p->total_q == 0) return SKV_OK;  // no query rows: nothing to launch
  if (plan_d == nullptr || info->num_ctas < 1 ||
      info->cta_offset < 16LL * info->num_work + 4LL * info->num_merge_rows)
    return SKV_ERR_INVALID;
  if (!p->o || (p->total_kv > 0 && (!p->k || !p->v))) return SKV_ERR_INVALID;
  const int32_t rows[3] = {p->total_q, p->total_kv, p->total_kv};
  const int32_t head_count[3] = {p->num_qo_heads, p->num_kv_heads, p->num_kv_heads};
  const void* base[3] = {p->q, p->k, p->v};
  const int64_t* stride[3] = {p->q_stride, p->k_stride, p->v_stride};
  for (int i = 0; i < 3; ++i) {
    if (rows[i] == 0) continue;
    if (base[i] == nullptr) return SKV_ERR_INVALID;
    if (!aligned16(base[i])) return SKV_ERR_ALIGNMENT;
    const int32_t count[2] = {rows[i], head_count[i]};
    for (int d = 0; d < 2; ++d) {
      if (count[d] <= 1) continue;  // never used
      if (stride[i][d] <= 0) return SKV_ERR_INVALID;
      if (stride[i][d] % 8 != 0) return SKV_ERR_ALIGNMENT;
      if (stride[i][d] >= (1LL << 38)) return SKV_ERR_UNSUPPORTED;  // 2^40 bytes: the tensor map's limit
    }
  }
  if (!aligned16(p->o) || !aligned16(p->o_part)) return SKV_ERR_ALIGNMENT;
  if (info->num_partial_rows > 0 && (!p->o_part || !p->lse_part)) return SKV_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int e = launch_prompt_attn(*p, reinterpret_cast<const PromptItem*>(plan_d), plan_d + info->cta_offset,
                                   info->num_ctas, s);
  if (e != 0 || info->num_merge_rows == 0) return cuda_status(e);
  const MergeItem* merges = reinterpret_cast<const MergeItem*>(plan_d + 16LL * info->num_work);
  return cuda_status(launch_merge(p->o_part, p->lse_part, nullptr, 0, merges, info->num_merge_rows, p->num_qo_heads,
                                  p->head_dim, p->o, p->o_dtype, p->lse, s));
}

}  // extern "C"
