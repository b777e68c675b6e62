// Rotary positions applied to queries and keys in one launch.
//
// x'_a = m (x_a cos t - x_b sin t), x'_b = m (x_a sin t + x_b cos t), t = position * inv_freq[pair].
// HBM-bound: every value is read and written once.  A block takes W tokens, forms their (cos, sin)
// tables once in shared memory (W * dim/2 sincos for W * (Hq + Hk) * dim/2 rotations) and streams
// the tokens' head rows through its threads, each holding one 16-value item of a row; the loads of
// kAhead rows are issued before the first is turned.  16384 tokens of 32 + 8 heads of 128: 62 us, 5.4 TB/s
// (84 % of the copy rate; 76 us with 16 consecutive values a thread); 64 tokens of 64 + 8 heads: 3.8 us.
#include "rope.cuh"

#include <algorithm>

namespace skv {

namespace {

using rope::Freq;

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // tokens per block
constexpr int kAhead = 2;       // rows each thread has in flight

struct RopeArgs {
  const void* q;
  const void* k;
  void* qo;
  void* ko;
  int64_t qs0, qs1, ks0, ks1, qo0, qo1, ko0, ko1;
  const int32_t* positions;
  int tokens, hq, hk, head_dim, items, per_block;
  Freq f;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float4 table[];
  __shared__ int32_t pos[kMaxTokens];
  __shared__ uint64_t turns[rope::kMaxPairs];
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * a.per_block, n = min(a.per_block, a.tokens - t0);
  const int nrot = a.f.dim / 16, stride4 = rope::table_float4s(a.f.dim);
  const int rows_per_pass = kThreads / a.items;
  const int item = tid % a.items;
  const rope::Item it = rope::item_of(item, a.f.dim, a.head_dim);
  const int heads = a.hq + a.hk;
  const int row = tid / a.items;
  const bool active = row < rows_per_pass;

  // the first rows' loads go out before the table is formed
  int tok = row / heads, h = row - tok * heads;
  auto src = [&](int tk, int hd) {
    return hd < a.hq ? static_cast<const T*>(a.q) + (int64_t)(t0 + tk) * a.qs0 + (int64_t)hd * a.qs1
                     : static_cast<const T*>(a.k) + (int64_t)(t0 + tk) * a.ks0 + (int64_t)(hd - a.hq) * a.ks1;
  };
  auto dst = [&](int tk, int hd) {
    return hd < a.hq ? static_cast<T*>(a.qo) + (int64_t)(t0 + tk) * a.qo0 + (int64_t)hd * a.qo1
                     : static_cast<T*>(a.ko) + (int64_t)(t0 + tk) * a.ko0 + (int64_t)(hd - a.hq) * a.ko1;
  };
  auto advance = [&](int& tk, int& hd) {
    hd += rows_per_pass;
    while (hd >= heads) {
      hd -= heads;
      ++tk;
    }
  };
  rope::Raw<T> raw[kAhead];
  int tks[kAhead], hds[kAhead];
  auto fetch = [&]() {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      tks[u] = tok;
      hds[u] = h;
      if (active && tok < n) raw[u].load(src(tok, h), it);
      advance(tok, h);
    }
  };
  fetch();
  if (tid < n) pos[tid] = a.f.dim > 0 ? a.positions[t0 + tid] : 0;
  rope::stage_turns(turns, a.f, tid, kThreads);
  __syncthreads();
  rope::fill_table(table, pos, n, turns, a.f.dim, a.f.mscale, a.f.halves, tid, kThreads);
  __syncthreads();
  if (!active) return;
  while (tks[0] < n) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (tks[u] < n) {
        float x[16];
        raw[u].values(x);
        if (it.turned) rope::turn_item(x, table + tks[u] * stride4, item, nrot, a.f.halves);
        rope::store_item(dst(tks[u], hds[u]), it, x);
      }
    }
    fetch();
  }
}

template <typename T>
int launch(const RopeArgs& a, cudaStream_t s) {
  const int smem = a.per_block * a.f.dim * 4;  // <= 16 KB: below the default limit
  const int blocks = (int)(((int64_t)a.tokens + a.per_block - 1) / a.per_block);
  rope_kernel<T><<<blocks, kThreads, smem, s>>>(a);
  return (int)cudaGetLastError();
}

}  // namespace

int launch_rope(const skv_rope_params& p, cudaStream_t s) {
  RopeArgs a;
  memset(&a, 0, sizeof(a));
  a.q = p.q;
  a.k = p.k;
  a.qo = p.q_out;
  a.ko = p.k_out;
  a.qs0 = p.q_stride[0];
  a.qs1 = p.q_stride[1];
  a.ks0 = p.k_stride[0];
  a.ks1 = p.k_stride[1];
  a.qo0 = p.q_out_stride[0];
  a.qo1 = p.q_out_stride[1];
  a.ko0 = p.k_out_stride[0];
  a.ko1 = p.k_out_stride[1];
  a.positions = p.positions;
  a.tokens = p.num_tokens;
  a.hq = p.num_q_heads;
  a.hk = p.num_k_heads;
  a.head_dim = p.head_dim;
  rope::make_freq(p.rope, p.inverse != 0, &a.f);
  const bool in_place = (p.num_q_heads == 0 || p.q == p.q_out) && (p.num_k_heads == 0 || p.k == p.k_out);
  // in place, copied values stay where they are
  a.items = p.rope.dim / 16 + (in_place ? 0 : ((p.head_dim - p.rope.dim) / 8 + 1) / 2);
  if (a.items == 0) return 0;
  a.per_block = rope::tokens_per_block(p.num_tokens, (a.hq + a.hk) * a.items, kThreads, kMaxTokens, device_sm_count());
  return p.dtype == SKV_F32 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s);
}

}  // namespace skv
