// GQA attention over a paged cache held in 8 bits (e4m3 or int8 codes) with one fp32 scale for each
// block of tokens and KV head:  k = ks * code, v = vs * code,
//   s_t = sm_scale (q . kcode_t) ks_t,   O = sum_t softmax(s)_t vs_t vcode_t,   LSE = ln sum_t e^{s_t}.
// The scales leave both products: ks multiplies the finished scores, vs the softmax weights, so the
// matrix instructions run on the codes themselves, which f16 holds exactly (e4m3: 4 significant
// bits, 2^-9 .. 448; int8: integers, carried as subnormals).
//
// Bound by HBM: 2 Hk D bytes per token.  One CTA takes `hc` KV heads (the largest of 8, 4, 2, 1 that
// divides Hk) of a slice of the batch's tokens (persistent, slices cut equal by the planner), so a
// token's rows of those heads are read together.  Eight consumer warps each own one head and 32
// tokens of a shared-memory stage and keep their own running maximum, sum and O, merged across the
// warps of a head when a work item ends.  The ring of stages is filled
//   - by TMA (one warp, one box of min(page, tile) slots x hc heads per page and tensor) where the
//     page size divides the tile or is a multiple of it, is a multiple of 8, and blocks are whole
//     groups of 8 tokens (one scale per group and head is staged);
//   - else by cp.async from four warps (any page size, block size and 16-byte strides; one scale per
//     token and head).  64-request 64/8-head e4m3 decode: 209 us with blocks of 4 in pages of 16, 212
//     with pages of 1, 272 with pages of 12, against 103 by TMA (pages and blocks of 16, 6.2 TB/s):
//     address arithmetic for 4096 copies a stage holds the ring back.
// With several query tokens the consumers bind it: 4 tokens over 171 k int8 tokens in pages of 64, 32/8
// heads: 76 us (4.6 TB/s), issue slots 46 % busy, most of it widening and the softmax of 16 rows.
//
// Decode has few query rows per KV head (R = group x query tokens <= 16), far below the 128 rows of
// the tcgen05 shapes, and each code needs widening in registers anyway, so the products are
// m16n8k16 f16 MMAs whose operands come straight from registers: S[rows, tokens] = Q . K^T leaves
// its accumulators exactly where the A operand of O[rows, dims] += P . V wants them.
//   - K: lane (g, t) reads 16-byte chunks t and t + 4 of its token's row; the dims of a k-step are
//     permuted to what one lane holds, Q is loaded under the same permutation.
//   - V: a B operand pairs two tokens of one dim.  Lane (g, t) reads the same 16 dims of four tokens
//     and interleaves bytes of two tokens (one byte permute per two pairs) before widening; output
//     dims are permuted, and come out as runs of 16 for one lane.
//   - chunks are XOR-swizzled by token so that the eight lanes of a 128-byte wavefront hit
//     different banks, for K and V alike.
// Precision: Q (bf16) moves to f16 after a power-of-two scale per row (largest element to
// [2^14, 2^15): exact for every element of at least 2^-31 of the row's largest).  Weights w = p vs are
// formed in fp32 and go to f16 relative to the largest w that the row has among the warp's 32 tokens,
// masked ones left out (w / wmax x 2^14: 11 bits down to 2^-28 of wmax, then a 2^-39th of it), and the
// partial product is scaled by wmax in fp32.  So neither a block that a row does not see nor one that
// it hardly attends to costs another block bits, and a key that outweighs all others has the weight
// 2^14 exactly.  The divisor is the fp32 sum of the exact p: the rounded w do not tell p apart where
// vs is 0 or far below its neighbours'.  (The maximum is raised once a score passes it by 2^8: p <= 2^8.)
#include <cudaTypedefs.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <string.h>

#include <algorithm>
#include <mutex>

#include "tc_ptx.cuh"

namespace skv {

namespace {

constexpr int kConsumers = 8;                 // warps
constexpr int kCopyWarps = 4;                 // producer warps (with TMA the last three only exit)
constexpr int kThreads = 32 * (kConsumers + kCopyWarps);
// Registers: 384 threads start with 168; the consumers take 208, the producers' warpgroup gives up to 88.
constexpr int kConsumerRegs = 208, kProducerRegs = 88;
static_assert(256 * kConsumerRegs + 128 * kProducerRegs <= kThreads * 168, "the split fits the launch's registers");
constexpr int kWarpTokens = 32;               // tokens of a stage that one consumer warp takes
constexpr float kRaise = 8.f;
constexpr float kTinyScale = 1.17549435e-38f;  // 2^-126
constexpr float kWeightTop = 16384.f;         // a row's largest weight of 32 tokens in f16

template <int D>
struct Smem {
  static constexpr int rows = kConsumers * kWarpTokens;           // (head, token) rows of a stage
  static constexpr int kv = rows * D;                             // bytes of K (and of V)
  static constexpr int scales = rows * 4;                         // of K (and of V)
  static constexpr int stage = 2 * (kv + scales);
  static constexpr int stages = D == 128 ? 3 : 5;
  static constexpr int merge = stages * stage;                    // [4 warps][8 rows][D] floats
  static constexpr int stat = merge + 4 * 8 * D * 4;              // [4 warps][16 rows] float2 (m, l)
  static constexpr int bars = stat + 4 * 16 * 8;
  static constexpr int misc = bars + 2 * stages * 8;
  static constexpr int total = misc + 16;
};
static_assert(Smem<128>::stage % 1024 == 0 && Smem<64>::stage % 1024 == 0, "swizzled boxes start on 1024 bytes");
static_assert(Smem<128>::total + 1024 <= 232448 && Smem<64>::total + 1024 <= 232448, "227 KB opt-in shared memory");

struct SArgs {
  const __nv_bfloat16* q;
  int box_log2;       // TMA: slots of a box
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  int64_t k0, k1, k2, v0, v1, v2;
  int64_t ks0, ks1, ks2, vs0, vs1, vs2;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* last;
  const WorkItem* work;
  const int32_t* cta_indptr;
  int num_pages, page_size, block_tokens, hq, hk, g;
  int hc_log2;        // KV heads of a CTA
  int head_groups;    // hk / hc
  int row_groups;     // ceil(g / 16) when one token's rows exceed a tile, else 1
  float scale_log2;
  void* o;
  float* lse;
  float* o_part;
  float* lse_part;
  int32_t* status;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// this thread's earlier cp.asyncs arrive on the barrier when they have landed
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// d = a . b + (c0, c0 in row g; c1, c1 in row g + 8)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                         float c1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %11, %11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ float lds_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// Four codes -> two f16 pairs, exact.  An int8 code c becomes the subnormal f16 (c + 128) 2^-24 -- its
// biased byte under a zero byte, one permute for two codes -- and the products start from minus 128
// times the sum of the other operand (in 2^-24 units), which takes the bias out again.
constexpr float kI8Unit = 1.f / 16777216.f;
template <bool I8>
__device__ __forceinline__ uint32_t biased(uint32_t w) {
  return I8 ? w ^ 0x80808080u : w;
}
template <bool I8>
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {  // w: biased
  if constexpr (I8) {
    lo = __byte_perm(w, 0u, 0x4140);
    hi = __byte_perm(w, 0u, 0x4342);
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2f(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// (o0, o1) += (c0, c1) f in one packed instruction
__device__ __forceinline__ void fma_pair(float& o0, float& o1, float c0, float c1, float f) {
  asm("{\n\t.reg .b64 o, c, f;\n\tmov.b64 o, {%0, %1};\n\tmov.b64 c, {%2, %3};\n\tmov.b64 f, {%4, %4};\n\t"
      "fma.rn.f32x2 o, c, f, o;\n\tmov.b64 {%0, %1}, o;\n\t}"
      : "+f"(o0), "+f"(o1)
      : "f"(c0), "f"(c1), "f"(f));
}
// (a, b) *= (fa, fb) in one packed instruction
__device__ __forceinline__ void mul_pair(float& a, float& b, float fa, float fb) {
  asm("{\n\t.reg .b64 x, f;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 f, {%2, %3};\n\tmul.rn.f32x2 x, x, f;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(fa), "f"(fb));
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// Token of an 8-token group that column c of a score tile holds, and the swizzle of a token's row:
// chosen so that the lanes of one shared-memory wavefront hit different banks (see the top).
template <int D>
__device__ __forceinline__ constexpr int col_token(int c) {
  return D == 128 ? ((c & 1) << 2) | (c >> 1) : c;
}
template <int D>
__device__ __forceinline__ constexpr int swizzle(int tok) {
  return D == 128 ? tok & 7 : (tok >> 1) & 3;
}

struct Range {
  int t0, t1, tiles;
};
__device__ __forceinline__ Range item_range(const SArgs& a, const WorkItem& w, int tile_tokens) {
  Range r;
  const int len = request_len(a.kv_indptr, a.last, w.r, a.page_size);
  r.t0 = w.page_begin * a.page_size;
  // w.split holds the first query token's key limit (causal), or a limit beyond any length
  r.t1 = min(min(w.page_end * a.page_size, len), w.split + w.q_count - 1);
  r.tiles = r.t1 > r.t0 ? (r.t1 - r.t0 + tile_tokens - 1) / tile_tokens : 0;
  return r;
}

template <bool I8, int D, bool WIDE, bool TMA, typename OutT>
__global__ void __launch_bounds__(kThreads, 1)
gqa_scaled_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ SArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using S = Smem<D>;
  constexpr int kChunks = D / 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  tc::grid_launch_dependents();  // the merge pass may be scheduled; it waits for this grid
  const uint32_t sbase = tc::smem_u32(smem);
  const uint32_t bar0 = sbase + S::bars;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::misc);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S::stages + s); };
  if (tid == 0) {
    for (int s = 0; s < S::stages; ++s) {
      tc::mbar_init(full_bar(s), TMA ? 33 : 32 * kCopyWarps);  // TMA: its transaction and 32 lanes' scales
      tc::mbar_init(empty_bar(s), kConsumers);
    }
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  __syncthreads();

  const int unit = blockIdx.x % (a.head_groups * a.row_groups), cta = blockIdx.x / (a.head_groups * a.row_groups);
  const int hc = 1 << a.hc_log2, h0 = (unit % a.head_groups) * hc, row0 = (unit / a.head_groups) * 16;
  const int tile_tokens = (kConsumers * kWarpTokens) >> a.hc_log2;
  const int w_begin = a.cta_indptr[cta], w_end = a.cta_indptr[cta + 1];

  if (warp >= kConsumers) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    if constexpr (TMA) {
      if (warp != kConsumers) return;
      // ============================================================================= TMA producer
      // Lane i stages the scales of 8-token group i / hc for head i % hc; the lanes of head 0 whose
      // group begins a box issue that box's K and V.
      const int first = (lane >> a.hc_log2) * 8, hh = lane & (hc - 1);
      const int box = 1 << a.box_log2;
      const bool issues = hh == 0 && (first & (box - 1)) == 0;
      const uint64_t pol = tc::policy_evict_first();
      int it = 0;
      bool ok = true;
      if (lane == 0) {
        tc::prefetch_tmap(&kmap);
        tc::prefetch_tmap(&vmap);
      }
      for (int wi = w_begin; wi < w_end && ok; ++wi) {
        const WorkItem w = a.work[wi];
        const Range rg = item_range(a, w, tile_tokens);
        const int32_t* ids = a.kv_indices + a.kv_indptr[w.r];
        auto page_of = [&](int tile) {  // page id of this lane's group, read one tile ahead of its use
          const int tok = rg.t0 + tile * tile_tokens + first;
          return tile < rg.tiles && tok < rg.t1 ? __ldg(ids + tok / a.page_size) : 0;
        };
        int next = page_of(0);
        for (int tile = 0; tile < rg.tiles; ++tile, ++it) {
          const int st = it % S::stages, page = next;
          const int tok = rg.t0 + tile * tile_tokens + first, slot = tok % a.page_size;
          const bool some = tok < rg.t1;
          const bool sound = (unsigned)page < (unsigned)a.num_pages;
          if (some && !sound && hh == 0) report(a.status, SKV_DEV_PAGE_OOB);
          next = page_of(tile + 1);
          if (it >= S::stages) ok = tc::mbar_wait(empty_bar(st), ((it / S::stages) + 1) & 1, abort_flag, a.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t kst = sbase + st * S::stage, vst = kst + S::kv, kss = vst + S::kv, vss = kss + S::scales;
          const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, issues && some));
          if (lane == 0) tc::mbar_arrive_expect_tx(full_bar(st), 2 * boxes * (uint32_t)((box * D) << a.hc_log2));
          __syncwarp();
          if (issues && some) {  // an id out of range reads as zeros
            const uint32_t at = (uint32_t)(first * D) << a.hc_log2;
            tc::tma_load_4d(kst + at, &kmap, full_bar(st), 0, slot, h0, page, pol);
            tc::tma_load_4d(vst + at, &vmap, full_bar(st), 0, slot, h0, page, pol);
          }
          const bool valid = some && sound;
          const int blk = slot / a.block_tokens;
          const int64_t so = (int64_t)(valid ? page : 0) * a.ks0 + (int64_t)blk * a.ks1 + (int64_t)(h0 + hh) * a.ks2;
          const int64_t vo = (int64_t)(valid ? page : 0) * a.vs0 + (int64_t)blk * a.vs1 + (int64_t)(h0 + hh) * a.vs2;
          const uint32_t dst = (uint32_t)((hh * (tile_tokens >> 3) + (first >> 3)) * 4);
          cp4(kss + dst, a.ks + (valid ? so : 0), valid);
          cp4(vss + dst, a.vs + (valid ? vo : 0), valid);
          cp_arrive(full_bar(st));
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!ok && lane == 0) {  // boxes in flight may still be landing: wait for them (bounded)
        for (int t = max(0, it - S::stages); t < it; ++t) {
          const uint64_t t_start = tc::globaltimer_ns();
          while (!tc::mbar_try_wait(full_bar(t % S::stages), (t / S::stages) & 1) &&
                 tc::globaltimer_ns() - t_start < 20000000ull) {
          }
        }
      }
      return;
    } else {
      // ======================================================================== cp.async producers
      const int pw = warp - kConsumers;
      const int mine = tile_tokens / kCopyWarps;  // 8, 16, 32 or 64 tokens of a tile for this warp
      int it = 0;
      bool ok = true;
      for (int wi = w_begin; wi < w_end && ok; ++wi) {
        const WorkItem w = a.work[wi];
        const Range rg = item_range(a, w, tile_tokens);
        const int32_t* ids = a.kv_indices + a.kv_indptr[w.r];
        // page ids of this warp's tokens, one tile ahead of their use
        int next[2];
        auto fetch_ids = [&](int tile) {
  #pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int tok = rg.t0 + tile * tile_tokens + pw * mine + b * 32 + lane;
            next[b] = (b * 32 + lane < mine && tok < rg.t1) ? __ldg(ids + tok / a.page_size) : 0;
          }
        };
        if (rg.tiles > 0) fetch_ids(0);
        for (int tile = 0; tile < rg.tiles; ++tile, ++it) {
          const int st = it % S::stages;
          int id[2] = {next[0], next[1]};
          if (tile + 1 < rg.tiles) fetch_ids(tile + 1);
          if (it >= S::stages) ok = tc::mbar_wait(empty_bar(st), ((it / S::stages) + 1) & 1, abort_flag, a.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t kst = sbase + st * S::stage, vst = kst + S::kv, kss = vst + S::kv, vss = kss + S::scales;
  #pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int n = min(32, mine - b * 32);
            if (n <= 0) break;
            const int first = pw * mine + b * 32;                       // tile-relative token of lane 0
            const int tok = rg.t0 + tile * tile_tokens + first + lane;
            bool valid = lane < n && tok < rg.t1;
            if (valid && (unsigned)id[b] >= (unsigned)a.num_pages) {
              report(a.status, SKV_DEV_PAGE_OOB);
              valid = false;
            }
            const int64_t page = valid ? id[b] : 0;
            const int slot = valid ? tok % a.page_size : 0, blk = slot / a.block_tokens;
            const int64_t ko = valid ? page * a.k0 + slot * a.k1 : -1;  // -1: zero-filled
            const int64_t vo = page * a.v0 + slot * a.v1;
            const int64_t kso = page * a.ks0 + blk * a.ks1, vso = page * a.vs0 + blk * a.vs1;
            const int copies = (n << a.hc_log2) * kChunks;              // a multiple of 32
  #pragma unroll 4
            for (int x = lane; x < copies; x += 32) {
              const int row = x / kChunks, c = x % kChunks, tl = row >> a.hc_log2, h = row & (hc - 1);
              const int64_t kx = __shfl_sync(0xffffffffu, ko, tl), vx = __shfl_sync(0xffffffffu, vo, tl);
              const int rt = first + tl;
              const uint32_t dst = (uint32_t)((h * tile_tokens + rt) * D + ((c ^ swizzle<D>(rt)) << 4));
              cp16(kst + dst, a.k + (kx < 0 ? 0 : kx + (int64_t)(h0 + h) * a.k2 + c * 16), kx >= 0);
              cp16(vst + dst, a.v + (kx < 0 ? 0 : vx + (int64_t)(h0 + h) * a.v2 + c * 16), kx >= 0);
            }
            const int pairs = n << a.hc_log2;
            for (int x0 = 0; x0 < pairs; x0 += 32) {
              const int x = x0 + lane, tl = x >> a.hc_log2, h = x & (hc - 1);
              const int64_t kx = __shfl_sync(0xffffffffu, ko, tl & 31);
              const int64_t sk = __shfl_sync(0xffffffffu, kso, tl & 31), sv = __shfl_sync(0xffffffffu, vso, tl & 31);
              if (x < pairs) {
                const uint32_t dst = (uint32_t)((h * tile_tokens + first + tl) * 4);
                cp4(kss + dst, a.ks + (kx < 0 ? 0 : sk + (int64_t)(h0 + h) * a.ks2), kx >= 0);
                cp4(vss + dst, a.vs + (kx < 0 ? 0 : sv + (int64_t)(h0 + h) * a.vs2), kx >= 0);
              }
            }
          }
          cp_arrive(full_bar(st));
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      return;
    }
  }

  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
  // ================================================================================== consumers
  const int g = lane >> 2, t = lane & 3;
  const int h = warp & (hc - 1), sub = warp >> a.hc_log2, subs = kConsumers >> a.hc_log2;
  const int kh = h0 + h;
  constexpr int kKSteps = D / 16;      // k-steps of Q . K^T
  constexpr int kDims = D / 8;         // dims of O each lane column covers (n-tiles of P . V)
  constexpr int kRowSets = WIDE ? 2 : 1;
  constexpr int kTokScales = TMA ? 1 : 2;  // scales of a lane's two tokens of an 8-token group
  // byte offset of the warp's 8-token groups in K (and V) of a stage, and of its scales
  uint32_t group_at[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int rt = sub * kWarpTokens + 8 * n;
    const int in = rt & ((1 << a.box_log2) - 1), box = rt >> a.box_log2;  // TMA: [box][head][slot]
    group_at[n] = (uint32_t)((TMA ? (((box << a.hc_log2) + h) << a.box_log2) + in : h * tile_tokens + rt) * D);
  }
  const uint32_t scale_at = 4u * (TMA ? h * (tile_tokens >> 3) + sub * 4 : h * tile_tokens + sub * kWarpTokens);
  int it = 0;
  bool ok = true;
  for (int wi = w_begin; wi < w_end; ++wi) {
    const WorkItem w = a.work[wi];
    const Range rg = item_range(a, w, tile_tokens);
    const int rows = w.q_count * a.g - row0;
    // rows g and g + 8 of the tile: query token, head, key limit
    int qi[2], qh[2], limit[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int r = g + 8 * s, rr = min(r, max(rows - 1, 0)) + row0;
      qi[s] = rr / a.g;
      qh[s] = kh * a.g + rr - qi[s] * a.g;
      limit[s] = min(rg.t1, w.split + qi[s]);
    }
    // every row of the warp sees keys below this one
    int all_see = min(limit[0], limit[1]);
#pragma unroll
    for (int x = 16; x >= 4; x >>= 1) all_see = min(all_see, __shfl_xor_sync(0xffffffffu, all_see, x));

    // Q in f16 under the k permutation: k-step 4 j + s of chunk j holds dims 16 (4 j + t) + 4 s ..
    uint32_t qf[kKSteps][4];
    float sc[2], bias[2] = {0.f, 0.f};
    {
      float x[2][D / 4];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bool live = (WIDE || s == 0) && g + 8 * s < rows;
        const __nv_bfloat16* src = a.q + ((int64_t)(w.q_start + qi[s]) * a.hq + qh[s]) * D;
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (live) v = __ldg(reinterpret_cast<const uint4*>(src + (4 * j + t) * 16 + e * 8));
            const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[s][j * 16 + e * 8 + 2 * i] = bf16_lo(wd[i]);
              x[s][j * 16 + e * 8 + 2 * i + 1] = bf16_hi(wd[i]);
              mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(wd[i])), fabsf(bf16_hi(wd[i]))));
            }
          }
        mx = quad_max(mx);
        const int e = mx > 0.f ? max((int)(__float_as_uint(mx) >> 23) - 127, -100) : 14;
        const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
        sc[s] = fabsf(a.scale_log2) * __uint_as_float((uint32_t)(127 - 14 + e) << 23) * (I8 ? 1.f / kI8Unit : 1.f);
        const float by = a.scale_log2 < 0.f ? -up : up;  // factors of the scores stay >= 0
#pragma unroll
        for (int i = 0; i < D / 4; ++i) x[s][i] *= by;
      }
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks) {
        const int i = (ks >> 2) * 16 + (ks & 3) * 4;
        qf[ks][0] = pack_f16(x[0][i], x[0][i + 1]);
        qf[ks][1] = WIDE ? pack_f16(x[1][i], x[1][i + 1]) : 0u;
        qf[ks][2] = pack_f16(x[0][i + 2], x[0][i + 3]);
        qf[ks][3] = WIDE ? pack_f16(x[1][i + 2], x[1][i + 3]) : 0u;
      }
      if constexpr (I8) {  // what the bias of K adds to a row's scores, of the values as rounded to f16
#pragma unroll
        for (int r = 0; r < kRowSets; ++r) {
          float sum = 0.f;
#pragma unroll
          for (int ks = 0; ks < kKSteps; ++ks)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&qf[ks][2 * e + r]));
              sum += y.x + y.y;
            }
          bias[r] = -128.f * kI8Unit * quad_sum(sum);
        }
      }
    }

    float o[kDims][2 * kRowSets];  // [dim of the lane's run][row set x (column 2t, 2t + 1)]
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kDims; ++j)
#pragma unroll
      for (int x = 0; x < 2 * kRowSets; ++x) o[j][x] = 0.f;

    for (int tile = 0; tile < rg.tiles; ++tile, ++it) {
      const int st = it % S::stages;
      ok = tc::mbar_wait(full_bar(st), (it / S::stages) & 1, abort_flag, a.status) && ok;
      const int tb = rg.t0 + tile * tile_tokens + sub * kWarpTokens;  // first token of this warp
      if (ok && tb < rg.t1) {
        const uint32_t kst = sbase + st * S::stage, vst = kst + S::kv;
        const uint32_t kss = sbase + st * S::stage + 2 * S::kv + scale_at, vss = kss + S::scales;
        // ---- scores: 4 tiles of 8 tokens, their accumulator chains interleaved
        float s[4][4];
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint32_t kw[4][4];
          const int tok = col_token<D>(g);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const uint4 v = lds128(kst + group_at[n] + tok * D + (((4 * j + t) ^ swizzle<D>(tok)) << 4));
            kw[n][0] = biased<I8>(v.x);
            kw[n][1] = biased<I8>(v.y);
            kw[n][2] = biased<I8>(v.z);
            kw[n][3] = biased<I8>(v.w);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              uint32_t b0, b1;
              widen<I8>(kw[n][x], b0, b1);
              if (j == 0 && x == 0) mma16816(s[n], qf[0], b0, b1, bias[0], bias[1]);
              else mma16816(s[n], qf[4 * j + x], b0, b1);
            }
        }
        // ---- mask, maximum.  Scores stay unscaled: score = s * f, f = ks sc >= 0 (kept above 0, so that
        // a masked -inf stays one; at 1e-30 every score of the block is 0 in any case)
        const int ta = col_token<D>(2 * t), tc1 = col_token<D>(2 * t + 1);
        float vsc[4][kTokScales], f[kRowSets][4][kTokScales];
        float mx[2] = {-INFINITY, -INFINITY};
        if (tb + kWarpTokens > all_see) {
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int r = 0; r < kRowSets; ++r) {
              if (tb + 8 * n + ta >= limit[r]) s[n][2 * r] = -INFINITY;
              if (tb + 8 * n + tc1 >= limit[r]) s[n][2 * r + 1] = -INFINITY;
            }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
          for (int e = 0; e < kTokScales; ++e) {  // TMA: one scale for the 8 tokens
            const int at = TMA ? 4 * n : (8 * n + (e ? tc1 : ta)) * 4;
            const float ks = lds_f(kss + at);
            const float vs = lds_f(vss + at);
            vsc[n][e] = vs < kTinyScale ? 0.f : vs;  // subnormal scales count as 0
#pragma unroll
            for (int r = 0; r < kRowSets; ++r) f[r][n][e] = fmaxf(ks * sc[r], 1e-30f);
          }
#pragma unroll
          for (int r = 0; r < kRowSets; ++r) {
            if constexpr (kTokScales == 1)
              mx[r] = fmaxf(mx[r], fmaxf(s[n][2 * r], s[n][2 * r + 1]) * f[r][n][0]);
            else
              mx[r] = fmaxf(mx[r], fmaxf(s[n][2 * r] * f[r][n][0], s[n][2 * r + 1] * f[r][n][kTokScales - 1]));
          }
        }
        bool raise = false;
#pragma unroll
        for (int r = 0; r < kRowSets; ++r) {
          mx[r] = quad_max(mx[r]);
          raise |= mx[r] > m[r] + kRaise;
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int r = 0; r < kRowSets; ++r) {
            const float mn = mx[r] > m[r] + kRaise ? mx[r] : m[r];
            const float al = mn == m[r] ? 1.f : ex2f(m[r] - mn);
            l[r] *= al;
            m[r] = mn;
#pragma unroll
            for (int j = 0; j < kDims; ++j) {
              o[j][2 * r] *= al;
              o[j][2 * r + 1] *= al;
            }
          }
        }
        // ---- weights w = p vs and the row's largest; in f16 relative to it
        float wmax[2] = {0.f, 0.f}, wmul[kRowSets], vmul[kRowSets];
#pragma unroll
        for (int r = 0; r < kRowSets; ++r) {
          const float nm = m[r] == -INFINITY ? 0.f : -m[r];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float p0 = ex2f(fmaf(s[n][2 * r], f[r][n][0], nm));
            const float p1 = ex2f(fmaf(s[n][2 * r + 1], f[r][n][kTokScales - 1], nm));
            l[r] += p0 + p1;
            s[n][2 * r] = p0;
            s[n][2 * r + 1] = p1;
            mul_pair(s[n][2 * r], s[n][2 * r + 1], vsc[n][0], vsc[n][kTokScales - 1]);
            wmax[r] = fmaxf(wmax[r], fmaxf(s[n][2 * r], s[n][2 * r + 1]));
          }
          wmax[r] = quad_max(wmax[r]);
          wmul[r] = fminf(__fdividef(kWeightTop, wmax[r]), 1.f / kTinyScale);  // finite for wmax = 0
          vmul[r] = fmaxf(wmax[r] * (1.f / kWeightTop), kTinyScale) * (I8 ? 1.f / kI8Unit : 1.f);
        }
        uint32_t pf[2][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (r < kRowSets) mul_pair(s[n][2 * r], s[n][2 * r + 1], wmul[r % kRowSets], wmul[r % kRowSets]);
            pf[n >> 1][(n & 1) * 2 + r] = r < kRowSets ? pack_f16(s[n][2 * r], s[n][2 * r + 1]) : 0u;
          }
        // ---- O += P . V: per lane 16 (D = 128) or 8 dims of 8 tokens
        float unbias[2] = {0.f, 0.f};
        if constexpr (I8) {  // the sum of the rounded weights: a product with f16 ones
          float w1[4];
          mma16816(w1, pf[0], 0x3C003C00u, 0x3C003C00u, 0.f, 0.f);
          mma16816(w1, pf[1], 0x3C003C00u, 0x3C003C00u);
          unbias[0] = -128.f * kI8Unit * w1[0];
          unbias[1] = -128.f * kI8Unit * w1[2];
        }
        constexpr int kWords = D / 32;  // words of a lane's run of dims
        uint32_t vw[4][2][kWords];      // [8-token group][token of the pair][word]
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tok = e ? tc1 : ta;
            const uint32_t row = vst + group_at[n] + tok * D;
            if constexpr (D == 128) {
              const uint4 v = lds128(row + ((col_token<D>(g) ^ swizzle<D>(tok)) << 4));
              vw[n][e][0] = biased<I8>(v.x);
              vw[n][e][1] = biased<I8>(v.y);
              vw[n][e][2] = biased<I8>(v.z);
              vw[n][e][3] = biased<I8>(v.w);
            } else {
              const uint2 v = lds64(row + (((g >> 1) ^ swizzle<D>(tok)) << 4) + ((g & 1) << 3));
              vw[n][e][0] = biased<I8>(v.x);
              vw[n][e][1] = biased<I8>(v.y);
            }
          }
        if (TMA && !I8 && tb + kWarpTokens > rg.t1) {  // slots past the end may hold NaN, and 0 x NaN is not 0
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (tb + 8 * n + (e ? tc1 : ta) >= rg.t1)
#pragma unroll
                for (int q = 0; q < kWords; ++q) vw[n][e][q] = 0u;
        }
#pragma unroll
        for (int q = 0; q < kWords; ++q) {
          uint32_t b[4][4];  // [8-token group][dim]: pairs of tokens
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            widen<I8>(__byte_perm(vw[n][0][q], vw[n][1][q], 0x5140), b[n][0], b[n][1]);
            widen<I8>(__byte_perm(vw[n][0][q], vw[n][1][q], 0x7362), b[n][2], b[n][3]);
          }
          float c[4][4];
#pragma unroll
          for (int d = 0; d < 4; ++d) mma16816(c[d], pf[0], b[0][d], b[1][d], unbias[0], unbias[1]);
#pragma unroll
          for (int d = 0; d < 4; ++d) mma16816(c[d], pf[1], b[2][d], b[3][d]);
#pragma unroll
          for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int r = 0; r < kRowSets; ++r)
              fma_pair(o[4 * q + d][2 * r], o[4 * q + d][2 * r + 1], c[d][2 * r], c[d][2 * r + 1], vmul[r]);
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(empty_bar(st));
    }
#pragma unroll
    for (int r = 0; r < kRowSets; ++r) l[r] = quad_sum(l[r]);

    // ---- join the warps of a head: half of them hand over to the other half, until one is left
    float* mbuf = reinterpret_cast<float*>(smem + S::merge);
    float2* sbuf = reinterpret_cast<float2*>(smem + S::stat);
    for (int half = subs >> 1; half > 0; half >>= 1) {
      const bool gives = sub >= half && sub < 2 * half, takes = sub < half;
      const int place = (sub - (gives ? half : 0)) * hc + h;  // < 4
#pragma unroll
      for (int r = 0; r < kRowSets; ++r) {
        tc::named_bar_sync(1, 32 * kConsumers);
        float4* mine = reinterpret_cast<float4*>(mbuf + place * 8 * D) + lane;
        if (gives) {
          if (t == 0) sbuf[place * 16 + 8 * r + g] = make_float2(m[r], l[r]);
#pragma unroll
          for (int j = 0; j < kDims; j += 2)
            mine[(j >> 1) * 32] = make_float4(o[j][2 * r], o[j][2 * r + 1], o[j + 1][2 * r], o[j + 1][2 * r + 1]);
        }
        tc::named_bar_sync(1, 32 * kConsumers);
        if (takes) {
          const float2 ml = sbuf[place * 16 + 8 * r + g];
          const float mn = fmaxf(m[r], ml.x), base = mn == -INFINITY ? 0.f : mn;
          const float fa = ex2f(m[r] - base), fb = ex2f(ml.x - base);
          m[r] = mn;
          l[r] = l[r] * fa + ml.y * fb;
#pragma unroll
          for (int j = 0; j < kDims; j += 2) {
            const float4 x = mine[(j >> 1) * 32];
            o[j][2 * r] = o[j][2 * r] * fa + x.x * fb;
            o[j][2 * r + 1] = o[j][2 * r + 1] * fa + x.y * fb;
            o[j + 1][2 * r] = o[j + 1][2 * r] * fa + x.z * fb;
            o[j + 1][2 * r + 1] = o[j + 1][2 * r + 1] * fa + x.w * fb;
          }
        }
      }
    }
    if (sub != 0) continue;
    // ---- write: column 2t holds dims d0 .., column 2t + 1 dims d1 .. of the rows
    const int d0 = D == 128 ? 16 * t : 16 * t, d1 = D == 128 ? 64 + 16 * t : 16 * t + 8;
#pragma unroll
    for (int r = 0; r < kRowSets; ++r) {
      if (g + 8 * r >= rows) continue;
      const float inv = l[r] > 0.f || l[r] != l[r] ? 1.f / l[r] : 0.f;
      const float lse = l[r] > 0.f || l[r] != l[r] ? (m[r] + log2f(l[r])) * kLn2 : -INFINITY;
      if (w.part_row < 0) {
        const int64_t at = (int64_t)(w.q_start + qi[r]) * a.hq + qh[r];
        if (t == 0 && a.lse != nullptr) a.lse[at] = lse;
        OutT* dst = reinterpret_cast<OutT*>(a.o) + at * D;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < kDims; j += 8) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = o[j + e][2 * r + c] * inv;
            OutT* p = dst + (c ? d1 : d0) + j;
            if constexpr (sizeof(OutT) == 4) {
              reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
              reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
            } else {
              uint4 u;
              __nv_bfloat162 h2[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) h2[e] = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
              u.x = *reinterpret_cast<uint32_t*>(&h2[0]);
              u.y = *reinterpret_cast<uint32_t*>(&h2[1]);
              u.z = *reinterpret_cast<uint32_t*>(&h2[2]);
              u.w = *reinterpret_cast<uint32_t*>(&h2[3]);
              *reinterpret_cast<uint4*>(p) = u;
            }
          }
      } else {
        const int64_t at = ((int64_t)w.part_row + (int64_t)qi[r] * w.part_stride) * a.hq + qh[r];
        if (t == 0) a.lse_part[at] = lse;
        float* dst = a.o_part + at * D;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < kDims; j += 4)
            *reinterpret_cast<float4*>(dst + (c ? d1 : d0) + j) =
                make_float4(o[j][2 * r + c] * inv, o[j + 1][2 * r + c] * inv, o[j + 2][2 * r + c] * inv,
                            o[j + 3][2 * r + c] * inv);
      }
    }
  }
}

struct Maps {
  CUtensorMap k, v;
};

template <bool I8, int D, bool WIDE, bool TMA, typename OutT>
int launch_s(const Maps& m, const SArgs& a, int ctas, cudaStream_t s) {
  static DeviceSmemAttr attr;
  const int smem = Smem<D>::total + 1024;
  const auto kernel = gqa_scaled_kernel<I8, D, WIDE, TMA, OutT>;
  if (const int e = attr.ensure(reinterpret_cast<const void*>(kernel), smem)) return e;
  kernel<<<ctas * a.head_groups * a.row_groups, kThreads, smem, s>>>(m.k, m.v, a);
  return (int)cudaGetLastError();
}
template <bool I8, int D, bool WIDE>
int launch_o(const Maps& m, const SArgs& a, int ctas, bool tma, int o_dtype, cudaStream_t s) {
  if (o_dtype == SKV_BF16)
    return tma ? launch_s<I8, D, WIDE, true, __nv_bfloat16>(m, a, ctas, s)
               : launch_s<I8, D, WIDE, false, __nv_bfloat16>(m, a, ctas, s);
  return tma ? launch_s<I8, D, WIDE, true, float>(m, a, ctas, s) : launch_s<I8, D, WIDE, false, float>(m, a, ctas, s);
}
template <bool I8>
int launch_d(const Maps& m, const SArgs& a, int ctas, int head_dim, bool wide, bool tma, int o_dtype, cudaStream_t s) {
  if (head_dim == 128)
    return wide ? launch_o<I8, 128, true>(m, a, ctas, tma, o_dtype, s)
                : launch_o<I8, 128, false>(m, a, ctas, tma, o_dtype, s);
  return wide ? launch_o<I8, 64, true>(m, a, ctas, tma, o_dtype, s)
              : launch_o<I8, 64, false>(m, a, ctas, tma, o_dtype, s);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Codes [page, slot, head, D] with caller strides (bytes); boxes of `box` slots x `hc` heads of one
// page, swizzled as the consumers read them (128-byte rows: by token % 8; 64-byte rows: token / 2 % 4).
bool cache_map(CUtensorMap* m, const void* base, const skv_paged_params& p, const int64_t* stride, int box, int hc) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)p.head_dim, (cuuint64_t)p.page_size, (cuuint64_t)p.num_kv_heads,
                              (cuuint64_t)std::max(1, p.num_pages)};
  cuuint64_t st[3];  // slot, head, page; a dimension of one entry never uses its stride
  st[0] = p.page_size > 1 ? (cuuint64_t)stride[1] : (cuuint64_t)p.head_dim;
  st[1] = p.num_kv_heads > 1 ? (cuuint64_t)stride[2] : (cuuint64_t)p.head_dim;
  st[2] = p.num_pages > 1 ? (cuuint64_t)stride[0] : (cuuint64_t)p.head_dim;
  for (cuuint64_t x : st)
    if (x == 0 || x >= (1ull << 40)) return false;
  const cuuint32_t bx[4] = {(cuuint32_t)p.head_dim, (cuuint32_t)box, (cuuint32_t)hc, 1}, estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, st, bx, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, p.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Rows of one tile are (query token, head of the group): 8 when a request's rows fit, else 16; a
// group of more than 16 heads is cut into row groups that run as CTAs side by side.
int gqa_scaled_q_tile(int group, int max_q_len) {
  const int rows = (int64_t)group * max_q_len <= 8 ? 8 : 16;
  return std::max(1, rows / group);
}
int gqa_scaled_units(int num_kv_heads, int group) {
  int hc = 8;
  while (num_kv_heads % hc) hc >>= 1;
  return num_kv_heads / hc * ((group + 15) / 16);
}
int gqa_scaled_tile_tokens(int num_kv_heads) {
  int hc = 8;
  while (num_kv_heads % hc) hc >>= 1;
  return kConsumers * kWarpTokens / hc;
}

int launch_gqa_scaled(const skv_paged_scaled_params& sp, const WorkItem* work, const int32_t* cta_indptr, int num_ctas,
                      int q_tile, cudaStream_t s) {
  const skv_paged_params& p = sp.base;
  SArgs a;
  a.q = static_cast<const __nv_bfloat16*>(p.q);
  a.k = static_cast<const uint8_t*>(p.k_cache);
  a.v = static_cast<const uint8_t*>(p.v_cache);
  a.ks = sp.k_scale;
  a.vs = sp.v_scale;
  a.k0 = p.k_stride[0];
  a.k1 = p.k_stride[1];
  a.k2 = p.k_stride[2];
  a.v0 = p.v_stride[0];
  a.v1 = p.v_stride[1];
  a.v2 = p.v_stride[2];
  a.ks0 = sp.k_scale_stride[0];
  a.ks1 = sp.k_scale_stride[1];
  a.ks2 = sp.k_scale_stride[2];
  a.vs0 = sp.v_scale_stride[0];
  a.vs1 = sp.v_scale_stride[1];
  a.vs2 = sp.v_scale_stride[2];
  a.kv_indptr = p.kv_indptr;
  a.kv_indices = p.kv_indices;
  a.last = p.kv_last_page_len;
  a.work = work;
  a.cta_indptr = cta_indptr;
  a.num_pages = p.num_pages;
  a.page_size = p.page_size;
  a.block_tokens = sp.block_tokens;
  a.hq = p.num_qo_heads;
  a.hk = p.num_kv_heads;
  a.g = p.num_qo_heads / p.num_kv_heads;
  a.hc_log2 = 3;
  while (a.hk % (1 << a.hc_log2)) --a.hc_log2;
  a.head_groups = a.hk >> a.hc_log2;
  a.row_groups = (a.g + 15) / 16;
  a.scale_log2 = p.sm_scale * kLog2e;
  a.o = p.o;
  a.lse = p.lse;
  a.o_part = p.o_part;
  a.lse_part = p.lse_part;
  a.status = p.status;
  const bool wide = q_tile * a.g > 8;
  // TMA where a tile is whole boxes of one page each and every 8-token group lies in one block; a box
  // takes `tile` or `page_size` slots (both powers of two then)
  const int hc = 1 << a.hc_log2, tile = kConsumers * kWarpTokens / hc, box = std::min(p.page_size, tile);
  Maps m;
  memset(&m, 0, sizeof(m));
  bool tma = p.page_size % 8 == 0 && sp.block_tokens % 8 == 0 && tile % box == 0 && p.page_size % box == 0;
  tma = tma && cache_map(&m.k, p.k_cache, p, p.k_stride, box, hc) && cache_map(&m.v, p.v_cache, p, p.v_stride, box, hc);
  a.box_log2 = 0;
  while ((1 << a.box_log2) < box) ++a.box_log2;
  return p.kv_dtype == SKV_I8 ? launch_d<true>(m, a, num_ctas, p.head_dim, wide, tma, p.o_dtype, s)
                              : launch_d<false>(m, a, num_ctas, p.head_dim, wide, tma, p.o_dtype, s);
}

}  // namespace skv
