// New keys and values into the paged cache, with the rotation (and, for 8-bit caches, the
// quantisation) applied on the way, in one launch; queries can be rotated by the same launch.
//
// HBM-bound: each new row is read once and its cache row written once.  A new token's request is
// found on the device (a 32-way search of append_indptr per warp), so the launch depends on the
// padded row count alone and replays from a graph while lengths change.
//
// Caches without block scales (append_rows_kernel): a block of threads takes W tokens, forms their
// (cos, sin) tables in shared memory once for all heads, and streams their K, V and Q rows through
// its threads, one 16-value item of a row each.
//
// Block-scaled caches (append_blocks_kernel): the unit is a segment -- the new tokens of one
// request that fall into one scale block -- for four heads of K or of V: a warp owns a head, takes
// the maximum of its (rotated) rows, settles the scale, re-encodes the block's other codes if the
// scale grew, then encodes the new rows.  Segments of up to 4 rows per lane stay in registers
// between the two passes; longer ones are read again from L1 / L2.  One owner per (block, head):
// no atomics, results do not depend on order.  Window w of the grid takes the segments that begin
// among its rows; the last blocks of the grid rotate Q.
#include "rope.cuh"

#include <cuda_fp8.h>

#include <algorithm>

namespace skv {

namespace {

using rope::Freq;

constexpr int kRowThreads = 256;
constexpr int kBlockThreads = 128;
constexpr int kMaxTokens = 16;   // tokens per block of threads, row kernel
constexpr int kTableTokens = 64; // tokens whose tables are held at once, block kernel
constexpr int kKeep = 4;         // items each lane holds between the two passes

enum CacheMode { MODE_BF16 = 0, MODE_E4M3 = 1, MODE_NONE = 2 };

struct AppendArgs {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* q;
  __nv_bfloat16* qo;
  uint8_t* kc;
  uint8_t* vc;
  float* ksc;
  float* vsc;
  int64_t k0, k1, v0, v1, q0, q1, qo0, qo1;
  int64_t kc0, kc1, kc2, vc0, vc1, vc2;  // cache strides in elements
  int64_t ks0, ks1, ks2, vs0, vs1, vs2;
  const int32_t* ip;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* last;
  const int32_t* positions;
  int32_t* status;
  int batch, num_rows, num_pages, page_size, hk, hq, head_dim, block_tokens;
  int per_block;        // rows of a window
  int num_windows, num_head_groups, num_kv_blocks;
  float inv_scale;
  Freq f;
};

// Warp-collective: the request of row t (the last r with ip[r] <= t), for ip[0] <= t < ip[batch].
__device__ __forceinline__ int find_request(const int32_t* ip, int batch, int t, int lane) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int64_t idx = lo + (int64_t)(lane + 1) * step;
    const bool le = idx < hi && __ldg(ip + idx) <= t;
    lo += __popc(__ballot_sync(0xffffffffu, le)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Where row t goes (warp-collective).  ok: the row belongs to a request of a sound table; page < 0:
// its page id is out of range.
struct Place {
  int r, i, n, pos, page;
  bool ok;
};
__device__ __forceinline__ Place find_place(const AppendArgs& a, int t, int lane) {
  Place pl;
  pl.r = find_request(a.ip, a.batch, t, lane);
  const int row0 = __ldg(a.ip + pl.r);
  pl.i = t - row0;
  pl.n = __ldg(a.ip + pl.r + 1) - row0;
  const int p0 = __ldg(a.kv_indptr + pl.r), np = __ldg(a.kv_indptr + pl.r + 1) - p0;
  const int64_t len = np > 0 ? (int64_t)(np - 1) * a.page_size + __ldg(a.last + pl.r) : 0;
  const int64_t pos = len - pl.n + pl.i;
  pl.pos = (int)pos;
  pl.page = -1;
  pl.ok = pl.i >= 0 && pl.i < pl.n && len >= pl.n && pos / a.page_size < np;
  if (pl.ok) {
    const int page = __ldg(a.kv_indices + (int64_t)p0 + pl.pos / a.page_size);
    if ((unsigned)page < (unsigned)a.num_pages) pl.page = page;
    else if (lane == 0) report(a.status, SKV_DEV_PAGE_OOB);
  } else if (lane == 0) {
    report(a.status, SKV_DEV_PLAN_BAD);
  }
  return pl;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ uint32_t i8_code(float x) {  // rn, [-127, 127], NaN -> 0
  const int c = __float2int_rn(fminf(fmaxf(x, -127.f), 127.f));
  return (uint32_t)(x == x ? c : 0) & 0xFFu;
}
template <bool I8>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  if constexpr (I8) return i8_code(a) | (i8_code(b) << 8) | (i8_code(c) << 16) | (i8_code(d) << 24);
  else return e4m3x4(a, b, c, d);
}
// An item's 16 codes: 8 bytes for each chunk.
template <bool I8>
__device__ __forceinline__ void store_codes(uint8_t* row, const rope::Item& it, const float (&x)[16], float inv) {
  float y[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) y[j] = x[j] * inv;
  *reinterpret_cast<uint2*>(row + it.c0) =
      make_uint2(codes4<I8>(y[0], y[1], y[2], y[3]), codes4<I8>(y[4], y[5], y[6], y[7]));
  *reinterpret_cast<uint2*>(row + it.c1) =
      make_uint2(codes4<I8>(y[8], y[9], y[10], y[11]), codes4<I8>(y[12], y[13], y[14], y[15]));
}

// Block-wide: rows [t0, t0 + n) of K and V into a cache without block scales (MODE_NONE: neither)
// and of Q, tables in `table`.
template <int MODE, int THREADS>
__device__ __forceinline__ void rows_pass(const AppendArgs& a, int t0, int n, float4* table) {
  __shared__ int32_t s_pos[kMaxTokens], s_page[kMaxTokens], s_slot[kMaxTokens], s_ok[kMaxTokens];
  const int tid = threadIdx.x, lane = tid & 31;
  const int total = min(a.num_rows, __ldg(a.ip + a.batch));
  n = min(n, total - t0);
  if (n <= 0) return;  // rows behind the last request
  const int items = a.head_dim / 16, nrot = a.f.dim / 16, stride4 = rope::table_float4s(a.f.dim);
  const int kv = MODE == MODE_NONE ? 0 : 2 * a.hk, heads = kv + a.hq;
  const int rows_per_pass = THREADS / items;
  const int item = tid % items;
  const rope::Item it = rope::item_of(item, a.f.dim, a.f.halves, a.head_dim);
  auto src = [&](int tk, int h) {
    const int64_t t = t0 + tk;
    return h < kv ? (h < a.hk ? a.k + t * a.k0 + (int64_t)h * a.k1 : a.v + t * a.v0 + (int64_t)(h - a.hk) * a.v1)
                  : a.q + t * a.q0 + (int64_t)(h - kv) * a.q1;
  };
  int tok = (tid / items) / heads, h = (tid / items) - tok * heads;
  rope::Raw<__nv_bfloat16> raw;
  if (tok < n) raw.load(src(tok, h), it);  // in flight while places and tables are formed
  for (int j = tid >> 5; j < n; j += THREADS / 32) {
    const Place pl = find_place(a, t0 + j, lane);
    if (lane == 0) {
      s_pos[j] = a.positions != nullptr ? __ldg(a.positions + t0 + j) : pl.pos;
      s_page[j] = pl.page;
      s_slot[j] = pl.pos % a.page_size;
      s_ok[j] = pl.ok;
    }
  }
  __syncthreads();
  rope::fill_table(table, s_pos, n, a.f, tid, THREADS);
  __syncthreads();
  while (tok < n) {
    const int tk = tok, hd = h;
    float x[16];
    raw.values(x);
    h += rows_per_pass;
    while (h >= heads) {
      h -= heads;
      ++tok;
    }
    if (tok < n) raw.load(src(tok, h), it);
    if (!s_ok[tk]) continue;
    const bool is_v = hd >= a.hk && hd < kv;
    if (it.turned && !is_v) rope::turn_item(x, table + tk * stride4, item, nrot, a.f.halves);
    if (hd >= kv) {
      rope::store_item(a.qo + (int64_t)(t0 + tk) * a.qo0 + (int64_t)(hd - kv) * a.qo1, it, x);
    } else if (MODE != MODE_NONE && s_page[tk] >= 0) {
      const int64_t off = is_v ? (int64_t)s_page[tk] * a.vc0 + (int64_t)s_slot[tk] * a.vc1 + (int64_t)(hd - a.hk) * a.vc2
                               : (int64_t)s_page[tk] * a.kc0 + (int64_t)s_slot[tk] * a.kc1 + (int64_t)hd * a.kc2;
      uint8_t* base = is_v ? a.vc : a.kc;
      if constexpr (MODE == MODE_BF16) rope::store_item(reinterpret_cast<__nv_bfloat16*>(base) + off, it, x);
      else store_codes<false>(base + off, it, x, a.inv_scale);
    }
  }
}

template <int MODE>
__global__ void __launch_bounds__(kRowThreads) append_rows_kernel(const __grid_constant__ AppendArgs a) {
  extern __shared__ float4 table[];
  const int t0 = blockIdx.x * a.per_block;
  rows_pass<MODE, kRowThreads>(a, t0, min(a.per_block, a.num_rows - t0), table);
}

// One segment of one head, by one warp: rows [t0, t0 + cnt) of `src` into slots [slot0, ...) of the
// block whose first slot is slot0 - old.  Block-wide barriers when TURN (table refills), so every
// warp of the block calls it; `live` is false for warps without a head.
template <bool I8, bool TURN>
__device__ __forceinline__ void segment(const AppendArgs& a, const __nv_bfloat16* src, int64_t s0, uint8_t* dst,
                                        int64_t d1, float* scale, int t0, int cnt, int old, int pos, bool live,
                                        float4* table, int32_t* s_pos) {
  const int tid = threadIdx.x, lane = tid & 31;
  const int items = a.head_dim / 16, item = lane % items, lt = 32 / items, sub = lane / items;
  const int nrot = a.f.dim / 16, stride4 = rope::table_float4s(a.f.dim);
  const rope::Item it = rope::item_of(item, a.f.dim, a.f.halves, a.head_dim);
  rope::Raw<__nv_bfloat16> raw[kKeep];
  const int step = lt * kKeep;  // tokens the warp holds at once
  const bool once = cnt <= step;
  float amax = 0.f, inv = 0.f;
  auto load = [&](int base, int end) {
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
      const int j = base + u * lt + sub;
      if (live && j < end) raw[u].load(src + (int64_t)(t0 + j) * s0, it);
    }
  };
  if (once) load(0, cnt);
  for (int pass = 0; pass < 2; ++pass) {
    for (int c0 = 0; c0 < cnt; c0 += kTableTokens) {
      const int cend = min(cnt, c0 + kTableTokens);
      if (TURN && (pass == 0 || cnt > kTableTokens)) {
        __syncthreads();  // the last table has been read
        for (int j = tid; j < cend - c0; j += kBlockThreads)
          s_pos[j] = a.positions != nullptr ? __ldg(a.positions + t0 + c0 + j) : pos + c0 + j;
        __syncthreads();
        rope::fill_table(table, s_pos, cend - c0, a.f, tid, kBlockThreads);
        __syncthreads();
      }
      for (int base = c0; base < cend; base += step) {
        if (!once) load(base, cend);
#pragma unroll
        for (int u = 0; u < kKeep; ++u) {
          const int j = base + u * lt + sub;
          if (!live || j >= cend) continue;
          float x[16];
          raw[u].values(x);
          if (TURN && it.turned) rope::turn_item(x, table + (j - c0) * stride4, item, nrot, a.f.halves);
          if (pass == 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
          } else {
            store_codes<I8>(dst + (int64_t)(old + j) * d1, it, x, inv);
          }
        }
      }
    }
    if (pass == 0 && live) {
      amax = warp_max(amax);
      const float before = old > 0 ? *scale : 0.f;
      float after = fmaxf(before, amax / (I8 ? 127.f : 448.f));
      if (after < 1.17549435e-38f) after = 0.f;
      inv = after > 0.f ? 1.f / after : 0.f;
      __syncwarp();  // every lane has read the old scale
      if (lane == 0) *scale = after;
      if (old > 0 && after > before) {
        for (int j = sub; j < a.block_tokens; j += lt) {  // the block's other slots, 16 codes a lane
          if (j >= old && j < old + cnt) continue;
          uint4* p = reinterpret_cast<uint4*>(dst + (int64_t)j * d1 + item * 16);
          const uint4 w = *p;
          uint32_t in[4] = {w.x, w.y, w.z, w.w}, out[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint32_t c = (in[e] >> (8 * b)) & 0xFFu;
              y[b] = (I8 ? (float)(int8_t)c : e4m3_to_float(c)) * before * inv;
            }
            out[e] = codes4<I8>(y[0], y[1], y[2], y[3]);
          }
          *p = make_uint4(out[0], out[1], out[2], out[3]);
        }
      }
    }
  }
}

template <bool I8>
__global__ void __launch_bounds__(kBlockThreads) append_blocks_kernel(const __grid_constant__ AppendArgs a) {
  extern __shared__ float4 table[];
  __shared__ int32_t s_pos[kTableTokens];
  const int b = blockIdx.x;
  if (b >= a.num_kv_blocks) {
    const int t0 = (b - a.num_kv_blocks) * a.per_block;
    rows_pass<MODE_NONE, kBlockThreads>(a, t0, min(a.per_block, a.num_rows - t0), table);
    return;
  }
  const int window = b % a.num_windows, part = b / a.num_windows;
  const bool is_v = part >= a.num_head_groups;
  const int h = (part - (is_v ? a.num_head_groups : 0)) * (kBlockThreads / 32) + (int)(threadIdx.x >> 5);
  const bool live = h < a.hk;
  const int lane = threadIdx.x & 31, bt = a.block_tokens;
  const int total = min(a.num_rows, __ldg(a.ip + a.batch));
  const int t1 = min((window + 1) * a.per_block, total);
  for (int t = window * a.per_block; t < t1;) {
    const Place pl = find_place(a, t, lane);
    if (!pl.ok) {  // the rest of a malformed request (or of the table) is skipped
      if (pl.i < 0 || pl.i >= pl.n) return;
      t += pl.n - pl.i;
      continue;
    }
    const int in = pl.pos % bt;
    const int cnt = min(min(bt - in, pl.n - pl.i), total - t);
    if ((pl.i == 0 || in == 0) && pl.page >= 0) {
      const int slot = pl.pos % a.page_size - in, blk = slot / bt;  // the block's first slot, its number
      if (is_v) {
        segment<I8, false>(a, a.v + (int64_t)h * a.v1, a.v0,
                           a.vc + (int64_t)pl.page * a.vc0 + (int64_t)slot * a.vc1 + (int64_t)h * a.vc2, a.vc1,
                           a.vsc + (int64_t)pl.page * a.vs0 + (int64_t)blk * a.vs1 + (int64_t)h * a.vs2, t, cnt, in,
                           pl.pos, live, table, s_pos);
      } else if (a.f.dim > 0) {
        segment<I8, true>(a, a.k + (int64_t)h * a.k1, a.k0,
                          a.kc + (int64_t)pl.page * a.kc0 + (int64_t)slot * a.kc1 + (int64_t)h * a.kc2, a.kc1,
                          a.ksc + (int64_t)pl.page * a.ks0 + (int64_t)blk * a.ks1 + (int64_t)h * a.ks2, t, cnt, in,
                          pl.pos, live, table, s_pos);
      } else {
        segment<I8, false>(a, a.k + (int64_t)h * a.k1, a.k0,
                           a.kc + (int64_t)pl.page * a.kc0 + (int64_t)slot * a.kc1 + (int64_t)h * a.kc2, a.kc1,
                           a.ksc + (int64_t)pl.page * a.ks0 + (int64_t)blk * a.ks1 + (int64_t)h * a.ks2, t, cnt, in,
                           pl.pos, live, table, s_pos);
      }
    }
    t += cnt;
  }
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

}  // namespace

int launch_kv_append(const skv_append_params& p, cudaStream_t s) {
  AppendArgs a;
  memset(&a, 0, sizeof(a));
  a.k = static_cast<const __nv_bfloat16*>(p.k);
  a.v = static_cast<const __nv_bfloat16*>(p.v);
  a.q = static_cast<const __nv_bfloat16*>(p.q);
  a.qo = static_cast<__nv_bfloat16*>(p.q_out);
  a.kc = static_cast<uint8_t*>(p.k_cache);
  a.vc = static_cast<uint8_t*>(p.v_cache);
  a.ksc = p.k_scale;
  a.vsc = p.v_scale;
  a.k0 = p.k_row_stride[0];
  a.k1 = p.k_row_stride[1];
  a.v0 = p.v_row_stride[0];
  a.v1 = p.v_row_stride[1];
  a.q0 = p.q_stride[0];
  a.q1 = p.q_stride[1];
  a.qo0 = p.q_out_stride[0];
  a.qo1 = p.q_out_stride[1];
  a.kc0 = p.k_stride[0];
  a.kc1 = p.k_stride[1];
  a.kc2 = p.k_stride[2];
  a.vc0 = p.v_stride[0];
  a.vc1 = p.v_stride[1];
  a.vc2 = p.v_stride[2];
  a.ks0 = p.k_scale_stride[0];
  a.ks1 = p.k_scale_stride[1];
  a.ks2 = p.k_scale_stride[2];
  a.vs0 = p.v_scale_stride[0];
  a.vs1 = p.v_scale_stride[1];
  a.vs2 = p.v_scale_stride[2];
  a.ip = p.append_indptr;
  a.kv_indptr = p.kv_indptr;
  a.kv_indices = p.kv_indices;
  a.last = p.kv_last_page_len;
  a.positions = p.positions;
  a.status = p.status;
  a.batch = p.batch;
  a.num_rows = p.num_rows;
  a.num_pages = p.num_pages;
  a.page_size = p.page_size;
  a.hk = p.num_kv_heads;
  a.hq = p.num_q_heads;
  a.head_dim = p.head_dim;
  a.block_tokens = p.block_tokens;
  a.inv_scale = p.kv_dtype == SKV_E4M3 && p.block_tokens == 0 ? 1.f / p.kv_scale : 1.f;
  rope::make_freq(p.rope, false, &a.f);
  const int64_t sms = device_sm_count();
  // enough windows to fill the SMs several times over, then up to kMaxTokens rows in each
  a.per_block = (int)std::min<int64_t>(kMaxTokens, std::max<int64_t>(1, p.num_rows / (sms * 8)));
  const int table_bytes = a.f.dim * 4;  // of one token
  if (p.block_tokens == 0) {
    const int blocks = cdiv(p.num_rows, a.per_block), smem = a.per_block * table_bytes;
    if (p.kv_dtype == SKV_BF16) append_rows_kernel<MODE_BF16><<<blocks, kRowThreads, smem, s>>>(a);
    else append_rows_kernel<MODE_E4M3><<<blocks, kRowThreads, smem, s>>>(a);
    return (int)cudaGetLastError();
  }
  a.num_windows = cdiv(p.num_rows, a.per_block);
  a.num_head_groups = cdiv(p.num_kv_heads, kBlockThreads / 32);
  a.num_kv_blocks = a.num_windows * a.num_head_groups * 2;
  const int blocks = a.num_kv_blocks + (p.num_q_heads > 0 ? a.num_windows : 0);
  const int smem = std::max(a.per_block, std::min(p.block_tokens, kTableTokens)) * table_bytes;  // <= 32 KB
  if (p.kv_dtype == SKV_I8) append_blocks_kernel<true><<<blocks, kBlockThreads, smem, s>>>(a);
  else append_blocks_kernel<false><<<blocks, kBlockThreads, smem, s>>>(a);
  return (int)cudaGetLastError();
}

}  // namespace skv
