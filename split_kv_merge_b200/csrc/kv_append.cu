// New keys and values into the paged cache, with the rotation (and, for 8-bit caches, the
// quantisation) applied on the way, in one launch; queries can be rotated by the same launch.
//
// HBM-bound: each new row is read once and its cache row written once.  A new token's request is
// found on the device (a 32-way search of append_indptr per warp), so the launch depends on the
// padded row count alone and replays from a graph while lengths change.
//
// Caches without block scales (append_rows_kernel): a block of threads takes W tokens, forms their
// (cos, sin) tables in shared memory once for all heads, and streams their K, V and Q rows through
// its threads, one 16-value item of a row each.  18 k tokens, 8 heads of 128, bf16: 37 us (31 without
// rotation), 147 MB moved; e4m3 with one scale 38 us.
//
// Block-scaled caches (append_blocks_kernel): the unit is a segment -- the new tokens of one
// request that fall into one scale block -- of K or of V.  A block of eight warps forms the segment's
// (cos, sin) table once and goes through the heads, as many at a time as the segment's length leaves
// warps for (one warp a head up to 16 tokens of 128 values, four for 64; a lane holds up to four items
// of 16 values): take the maximum of the head's (rotated) rows, settle the scale, encode the rows from
// registers while the next heads' rows are on their way, re-encode the block's other codes if the scale
// grew.  Segments of more than 64 tokens are read twice.  One owner per (block, head): no atomics, results do not depend on order.  Window w
// of the grid takes the segments that begin among its rows; the last blocks of the grid rotate Q.
// (One warp per head, two passes over its rows: 93 us for 18 k tokens, 8 heads of 128, blocks of 64;
// eight warps for two heads, each with its own search and table: 121 us; sixteen warps a segment, one
// item a lane: 43 us, and 5.9 us for a step of 64 tokens; this form: 39 and 5.3 us.  A segment takes 13
// (V) to 20 us (K), two to an SM at a time: 1.4 us until its place is known, 4 for the table, then 3 us
// for every two heads.)
#include "rope.cuh"

#include <cuda_fp8.h>

#include <algorithm>

namespace skv {

namespace {

using rope::Freq;

constexpr int kRowThreads = 256;
constexpr int kBlockWarps = 8;   // block kernel
constexpr int kLaneRows = 4;     // rows of a chunk that a lane holds, block kernel
constexpr int kMaxPairs = 64;    // head_dim <= 128
constexpr int kMaxTokens = 16;   // tokens per block of threads, row kernel
constexpr int kTableTokens = 64; // tokens whose tables are held at once, block kernel

enum Turn { kCopy = 0, kInterleaved = 1, kHalves = 2 };
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
  int per_q_block;      // rows of a block of threads that rotates Q beside the block kernel
  int num_windows;
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

// Where row t goes (warp-collective).  ok: the row belongs to a request of a sound table.  The page
// id is as the table has it (checked by sound_page, so that its load can be in flight meanwhile).
struct Place {
  int i, n, pos, page;
  int64_t first_page;  // the request's first entry of kv_indices
  bool ok;
};
__device__ __forceinline__ Place find_place(const AppendArgs& a, int t, int lane) {
  Place pl;
  const int r = find_request(a.ip, a.batch, t, lane);
  const int row0 = __ldg(a.ip + r);
  pl.i = t - row0;
  pl.n = __ldg(a.ip + r + 1) - row0;
  const int p0 = __ldg(a.kv_indptr + r), np = __ldg(a.kv_indptr + r + 1) - p0;
  const int64_t len = np > 0 ? (int64_t)(np - 1) * a.page_size + __ldg(a.last + r) : 0;
  pl.first_page = p0;
  pl.page = -1;
  pl.ok = pl.i >= 0 && pl.i < pl.n && len >= pl.n && len <= (int64_t)np * a.page_size && len <= INT32_MAX;
  pl.pos = pl.ok ? (int)len - pl.n + pl.i : 0;
  if (pl.ok) pl.page = __ldg(a.kv_indices + (int64_t)p0 + pl.pos / a.page_size);
  else if (lane == 0) report(a.status, SKV_DEV_PLAN_BAD);
  return pl;
}
__device__ __forceinline__ bool sound_page(const AppendArgs& a, int page, int lane) {
  if ((unsigned)page < (unsigned)a.num_pages) return true;
  if (lane == 0) report(a.status, SKV_DEV_PAGE_OOB);
  return false;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
// An int8 code (rn, [-127, 127], NaN -> 0) in the low byte: 1.5 x 2^23 leaves a float's last bits integral.
// (The conversion instruction runs at a quarter of the rate: 47 us against 44 at the size above.)
__device__ __forceinline__ uint32_t i8_code(float x) {
  return __float_as_uint(fminf(fmaxf(x == x ? x : 0.f, -127.f), 127.f) + 12582912.f);
}
template <bool I8>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  if constexpr (I8)
    return __byte_perm(__byte_perm(i8_code(a), i8_code(b), 0x0040), __byte_perm(i8_code(c), i8_code(d), 0x0040), 0x5410);
  else return e4m3x4(a, b, c, d);
}
// An item's 16 codes: 8 bytes for each chunk.
template <bool I8>
__device__ __forceinline__ void encode_item(const float (&x)[16], float inv, uint2 (&code)[2]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float* y = x + 8 * c;
    code[c] = make_uint2(codes4<I8>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                         codes4<I8>(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
  }
}

// Block-wide: rows [t0, t0 + n) of K and V into a cache without block scales (MODE_NONE: neither)
// and of Q, tables in `table`.
template <int MODE, int THREADS>
__device__ __forceinline__ void rows_pass(const AppendArgs& a, int t0, int n, float4* table) {
  __shared__ int32_t s_pos[kMaxTokens], s_page[kMaxTokens], s_slot[kMaxTokens], s_ok[kMaxTokens];
  __shared__ uint64_t turns[kMaxPairs];
  const int tid = threadIdx.x, lane = tid & 31;
  const int total = min(a.num_rows, __ldg(a.ip + a.batch));
  n = min(n, total - t0);
  if (n <= 0) return;  // rows behind the last request
  const int items = a.head_dim / 16, nrot = a.f.dim / 16, stride4 = rope::table_float4s(a.f.dim);
  const int kv = MODE == MODE_NONE ? 0 : 2 * a.hk, heads = kv + a.hq;
  const int rows_per_pass = THREADS / items;
  const int item = tid % items;
  const rope::Item it = rope::item_of(item, a.f.dim, a.head_dim);
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
      s_page[j] = MODE != MODE_NONE && pl.ok && sound_page(a, pl.page, 0) ? pl.page : -1;
      s_slot[j] = pl.pos % a.page_size;
      s_ok[j] = pl.ok;
    }
  }
  rope::stage_turns(turns, a.f, tid, THREADS);
  __syncthreads();
  rope::fill_table(table, s_pos, n, turns, a.f.dim, a.f.mscale, a.f.halves, tid, THREADS);
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
      else {
        uint2 code[2];
        encode_item<false>(x, a.inv_scale, code);
        *reinterpret_cast<uint2*>(base + off + it.c0) = code[0];
        *reinterpret_cast<uint2*>(base + off + it.c1) = code[1];
      }
    }
  }
}

template <int MODE>
__global__ void __launch_bounds__(kRowThreads) append_rows_kernel(const __grid_constant__ AppendArgs a) {
  extern __shared__ float4 table[];
  const int t0 = blockIdx.x * a.per_block;
  rows_pass<MODE, kRowThreads>(a, t0, min(a.per_block, a.num_rows - t0), table);
}

// Shared memory of the block kernel beside the table.
struct BlockShared {
  uint64_t turns[kMaxPairs];
  int32_t pos[kTableTokens];
  uint32_t amax[2][kBlockWarps];
};

// K's or V's pointers (V is a constant of the caller: strides stay in the parameter bank).
template <bool V>
__device__ __forceinline__ const __nv_bfloat16* row_ptr(const AppendArgs& a, int t, int h) {
  return V ? a.v + t * a.v0 + h * a.v1 : a.k + t * a.k0 + h * a.k1;
}
template <bool V>
__device__ __forceinline__ uint8_t* cache_ptr(const AppendArgs& a, int page, int slot, int h) {
  return V ? a.vc + page * a.vc0 + slot * a.vc1 + h * a.vc2 : a.kc + page * a.kc0 + slot * a.kc1 + h * a.kc2;
}
template <bool V>
__device__ __forceinline__ float* scale_ptr(const AppendArgs& a, int page, int blk, int h) {
  return V ? a.vsc + page * a.vs0 + blk * a.vs1 + h * a.vs2 : a.ksc + page * a.ks0 + blk * a.ks1 + h * a.ks2;
}

// The codes of a block's slots outside [old, old + cnt), written again for a scale 1 / inv.
template <bool I8>
__device__ __noinline__ void reencode(uint8_t* dst, int64_t row, int tokens, int old, int cnt, int sub, int lanes, int item,
                                      float before, float inv) {
  for (int j = sub; j < tokens; j += lanes) {
    if (j >= old && j < old + cnt) continue;
    uint4* p = reinterpret_cast<uint4*>(dst + j * row + item * 16);
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

// One segment, by the whole block: rows [t0, t0 + cnt) into slots [first + old, ...) of the scale block
// `blk` of `page`, whose first slot is `first`; pos: the first row's position.  ONCE: the segment is one
// chunk of rows, which stay in the lanes' registers.
template <bool I8, bool V, int TURN, bool ONCE>
__device__ __forceinline__ void segment(const AppendArgs& a, int t0, int cnt, int page, int first, int blk, int old,
                                        int pos, float4* table, BlockShared& sh) {
  constexpr int threads = 32 * kBlockWarps;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = a.head_dim / 16, item = lane % items, lt = 32 / items;
  int g = 1;  // warps of a head
  while (g < kBlockWarps && min(cnt, kTableTokens) > g * lt * kLaneRows) g *= 2;
  const int part = warp & (g - 1), sub = part * lt + lane / items;  // this lane's first row of a chunk
  const int step = g * lt;  // rows between a lane's
  const int nrot = a.f.dim / 16, stride4 = rope::table_float4s(a.f.dim);
  const rope::Item it = rope::item_of(item, TURN == kCopy ? 0 : a.f.dim, a.head_dim);
  const int64_t src_row = V ? a.v0 : a.k0, dst_row = V ? a.vc1 : a.kc1;
  // this lane's row of the first chunk, for the head its warp begins with; heads follow by strides
  const int heads = kBlockWarps / g, h0 = warp / g;
  const __nv_bfloat16* src = row_ptr<V>(a, t0 + sub, h0);
  const int64_t src_head = heads * (V ? a.v1 : a.k1);
  rope::Raw<__nv_bfloat16> raw[kLaneRows];
  float x[kLaneRows][16];
  auto mine = [&](int c0, int i) { return sub + i * step < (ONCE ? cnt : min(cnt - c0, kTableTokens)); };
  auto load = [&](int c0) {
#pragma unroll
    for (int i = 0; i < kLaneRows; ++i)
      if (mine(c0, i)) raw[i].load(src + (c0 + i * step) * src_row, it);
  };
  auto fill = [&](int c0) {
    if (TURN == kCopy) return;
    const int n = min(cnt - c0, kTableTokens);
    __syncthreads();  // the last table has been read
    for (int j = tid; j < n; j += threads)
      sh.pos[j] = a.positions != nullptr ? __ldg(a.positions + t0 + c0 + j) : pos + c0 + j;
    __syncthreads();
    rope::fill_table(table, sh.pos, n, sh.turns, a.f.dim, a.f.mscale, TURN == kHalves, tid, threads);
    __syncthreads();
  };
  auto turn = [&](int c0, float top) {  // raw -> x, and the largest of them
#pragma unroll
    for (int i = 0; i < kLaneRows; ++i) {
      if (!mine(c0, i)) continue;
      raw[i].values(x[i]);
      if (TURN != kCopy && it.turned)
        rope::turn_item(x[i], table + (sub + i * step) * stride4, item, nrot, TURN == kHalves);
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[i][e]));
    }
    return top;
  };
  if (ONCE && h0 < a.hk) load(0);
  if (!sound_page(a, page, lane)) return;  // the same for every warp
  if (ONCE) fill(0);
  float* scale = scale_ptr<V>(a, page, blk, h0);
  const int64_t scale_head = heads * (V ? a.vs2 : a.ks2);
  uint8_t* dst = cache_ptr<V>(a, page, first, h0);
  const int64_t dst_head = heads * (V ? a.vc2 : a.kc2);
  auto store = [&](int c0, float inv) {
#pragma unroll
    for (int i = 0; i < kLaneRows; ++i) {
      if (!mine(c0, i)) continue;
      uint2 code[2];
      encode_item<I8>(x[i], inv, code);
      uint8_t* row = dst + (old + c0 + sub + i * step) * dst_row;
      *reinterpret_cast<uint2*>(row + it.c0) = code[0];
      *reinterpret_cast<uint2*>(row + it.c1) = code[1];
    }
  };
  int odd = 0;
#pragma unroll 1
  for (int h = h0; h < h0 + a.hk; h += heads, odd ^= 1) {  // the same number of rounds for every warp
    const bool live = h < a.hk;
    const float before = live && old > 0 ? *scale : 0.f;
    float top = 0.f;
    if constexpr (ONCE) {
      if (live) {
        top = turn(0, 0.f);
        src += src_head;
        if (h + heads < a.hk) load(0);  // the next heads' rows
      }
    } else {
#pragma unroll 1
      for (int c0 = 0; c0 < cnt; c0 += kTableTokens) {
        fill(c0);
        if (!live) continue;
        load(c0);
        top = turn(c0, top);
      }
    }
    uint32_t amax = __reduce_max_sync(0xffffffffu, __float_as_uint(top));  // of values >= 0: order as integers
    if (g > 1) {  // two buffers: the next heads' maxima are written while these are read
      if (lane == 0) sh.amax[odd][warp] = amax;
      __syncthreads();  // and every warp has read the old scale
      amax = __reduce_max_sync(0xffffffffu, sh.amax[odd][warp - part + (lane & (g - 1))]);
    }
    float after = fmaxf(before, __uint_as_float(amax) * (I8 ? 1.f / 127.f : 1.f / 448.f));
    if (after < 1.17549435e-38f) after = 0.f;
    const float inv = after > 0.f ? __fdividef(1.f, after) : 0.f;
    __syncwarp();
    if (live && lane == 0 && part == 0) *scale = after;
    if constexpr (ONCE) {
      if (live) store(0, inv);
    } else {
#pragma unroll 1
      for (int c0 = 0; c0 < cnt; c0 += kTableTokens) {
        fill(c0);
        if (!live) continue;
        load(c0);
        turn(c0, 0.f);
        store(c0, inv);
      }
      src += src_head;
    }
    if (live && old > 0 && after > before)
      reencode<I8>(dst, dst_row, a.block_tokens, old, cnt, sub, lt * g, item, before, inv);
    scale += scale_head;
    dst += dst_head;
  }
}

// The segments that begin in a window.  (K's and V's loops apart: one loop over both would keep both
// sets of strides in registers.  LONG: blocks may hold more than kTableTokens tokens.)
template <bool I8, bool V, int TURN, bool LONG>
__device__ __forceinline__ void window_segments(const AppendArgs& a, int window, float4* table, BlockShared& sh) {
  if (TURN != kCopy) rope::stage_turns(sh.turns, a.f, threadIdx.x, 32 * kBlockWarps);
  const int lane = threadIdx.x & 31, bt = a.block_tokens;
  const int total = min(a.num_rows, __ldg(a.ip + a.batch));
  const int t1 = (int)min((window + 1) * (int64_t)a.per_block, (int64_t)total);
  int t = window * a.per_block;
  if (t >= t1) return;
  Place pl = find_place(a, t, lane);
  while (true) {
    int cnt = pl.n - pl.i, page = pl.page;
    if (pl.ok) {
      const int in = pl.pos % bt;
      cnt = min(min(bt - in, cnt), total - t);
      // the request's next segment needs its page id only; that load runs beside this segment
      const bool more = pl.i + cnt < pl.n && t + cnt < t1;
      if (more) pl.page = __ldg(a.kv_indices + pl.first_page + (pl.pos + cnt) / a.page_size);
      if (pl.i == 0 || in == 0) {
        const int first = pl.pos % a.page_size - in;  // the block's first slot
        __syncthreads();  // the last segment's shared values have been read
        if (LONG && cnt > kTableTokens)
          segment<I8, V, TURN, false>(a, t, cnt, page, first, first / bt, in, pl.pos, table, sh);
        else
          segment<I8, V, TURN, true>(a, t, cnt, page, first, first / bt, in, pl.pos, table, sh);
      }
      t += cnt;
      if (more) {
        pl.i += cnt;
        pl.pos += cnt;
        continue;
      }
    } else {  // the rest of a malformed request (or of the table) is skipped
      if (pl.i < 0 || cnt <= 0) return;
      t += cnt;
    }
    if (t >= t1) return;
    pl = find_place(a, t, lane);
  }
}

template <bool I8, int TURN, bool LONG>
__global__ void __launch_bounds__(32 * kBlockWarps, 2) append_blocks_kernel(const __grid_constant__ AppendArgs a) {
  extern __shared__ float4 table[];
  __shared__ BlockShared sh;
  // K's windows first: they take longer (a table, rotation), so V's even out the launch's end
  const int b = blockIdx.x;
  if (b < a.num_windows) {
    window_segments<I8, false, TURN, LONG>(a, b, table, sh);
  } else if (b < 2 * a.num_windows) {
    window_segments<I8, true, kCopy, LONG>(a, b - a.num_windows, table, sh);
  } else {
    const int t0 = (b - 2 * a.num_windows) * a.per_q_block;
    rows_pass<MODE_NONE, 32 * kBlockWarps>(a, t0, min(a.per_q_block, a.num_rows - t0), table);
  }
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <bool I8, bool LONG>
int launch_turn(const AppendArgs& a, int blocks, int smem, cudaStream_t s) {
  constexpr int threads = 32 * kBlockWarps;
  if (a.f.dim == 0) append_blocks_kernel<I8, kCopy, LONG><<<blocks, threads, smem, s>>>(a);
  else if (a.f.halves) append_blocks_kernel<I8, kHalves, LONG><<<blocks, threads, smem, s>>>(a);
  else append_blocks_kernel<I8, kInterleaved, LONG><<<blocks, threads, smem, s>>>(a);
  return (int)cudaGetLastError();
}
template <bool I8>
int launch_blocks(const AppendArgs& a, int blocks, int smem, cudaStream_t s) {
  return a.block_tokens > kTableTokens ? launch_turn<I8, true>(a, blocks, smem, s)
                                       : launch_turn<I8, false>(a, blocks, smem, s);
}

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
  const int table_bytes = a.f.dim * 4;  // of one token
  const int items = a.head_dim / 16;
  if (p.block_tokens == 0) {
    a.per_block = rope::tokens_per_block(p.num_rows, (2 * a.hk + a.hq) * items, kRowThreads, kMaxTokens, sms);
    const int blocks = cdiv(p.num_rows, a.per_block), smem = a.per_block * table_bytes;
    if (p.kv_dtype == SKV_BF16) append_rows_kernel<MODE_BF16><<<blocks, kRowThreads, smem, s>>>(a);
    else append_rows_kernel<MODE_E4M3><<<blocks, kRowThreads, smem, s>>>(a);
    return (int)cudaGetLastError();
  }
  // windows of one row while there are few, then three an SM for each of K and V: two blocks are
  // resident, and the third evens out what segments of unlike lengths leave (two, three, four, five an
  // SM: 45.6, 40.6, 42.8, 44.9 us at the size that the top names; K's and V's windows in turns: 42.8)
  a.per_block = (int)std::max<int64_t>(1, p.num_rows / (sms * 3));
  a.num_windows = cdiv(p.num_rows, a.per_block);
  a.per_q_block = 1;
  int blocks = 2 * a.num_windows;
  if (a.hq > 0) {
    a.per_q_block = rope::tokens_per_block(p.num_rows, a.hq * items, 32 * kBlockWarps, kMaxTokens, sms);
    blocks += cdiv(p.num_rows, a.per_q_block);
  }
  const int smem = std::max(a.per_q_block, std::min(p.block_tokens, kTableTokens)) * table_bytes;  // <= 32 KB
  return p.kv_dtype == SKV_I8 ? launch_blocks<true>(a, blocks, smem, s) : launch_blocks<false>(a, blocks, smem, s);
}

}  // namespace skv
