// Attention over whole prompts: packed sequences of different lengths, grouped heads, causal or not,
// keys and values as the projections left them ([token, head, dim], any 16-byte strides).
//   s = sm_scale q . k,  O = softmax(s) v,  LSE = ln sum e^s;  with the causal mask the n query tokens
//   of a sequence of L keys are its last n positions, query token i sees keys t <= L - n + i.
//
// Bound by the tensor cores and the exponentials together: a 128 x 128 score tile costs two
// 128 x 128 x D products (1024 cycles at D = 128) and 16384 exponentials (1024 cycles at 16 per SM).
// Hence two query tiles per CTA, A and B, that take turns: while the softmax warps of A work on
// S_A, the tensor cores run P_B V and Q_B K^T.  A and B are two heads of one group on the same
// tokens (they share every K and V tile), or, for odd groups, consecutive 128-token tiles of a head.
//
// TMEM holds S_A, S_B (128 fp32 columns each) and O_A, O_B; P (bf16) overwrites the first half of its
// own S and is the A operand of P V straight from TMEM.  The MMAs of a query tile are issued by one
// thread and complete in order, so two facts need no barrier of their own: Q K^T of the next tile
// may overwrite S / P as soon as it is issued after P V, and a full S means the P V before it is
// done, so the softmax warps may rescale O.  A and B have an issuing warp each: an MMA of these
// shapes holds its issuer about 80 cycles (it runs for 64), a wait or commit after one some 200, and
// one issuer for both sides was busy 4130 cycles per pair of tiles (clock stamps of one CTA).  The two
// issue in strict turns: left to themselves A and B fall into step, both in the softmax and then both
// at the tensor cores (1214 us against 976 for that form, 4096 query tokens over 16384 keys, 32/8 heads).
// What is left is the chain of one side: 2100 cycles of softmax, its weights' way to the issuer, 1024 of
// MMAs, their scores' way back: 3800 for a pair of tiles, 2048 of them the tensor cores'.  Scores in two
// buffers of 64 keys, which break that chain, measured slower (1072 us on 951): a 128 x 64 x 16 product of two
// shared-memory operands takes 59 cycles, the one of 128 x 128 x 16 only 64.  Weights handed over in
// halves with the maximum taken beside the exponentials: 1005 us.  (These cycles are from before the sum of
// the rounded weights, which adds 4 % to the kernel: 920 -> 956 us.)
// The running maximum is raised only when a score passes it by 2^8, so O is rarely rescaled.
//
// Persistent: the planner hands every CTA a list of items (a pair of query tiles and a range of
// key tiles), longest first onto the least loaded.  Items of few rows over many keys, and a few of
// those that would make no full round, are cut along the keys into fp32 partials that the merge pass
// joins.  An item's end costs about 5000 cycles (the last P V, its results, the next item's first
// scores): its code runs once in a while and is kept short, and results leave by whole sectors (16
// sequences of 64 .. 2048 tokens: 194 us, 204 with 16-byte stores, 218 with all of it unrolled; now 203).
// Roles: warps 0-3 softmax of A, 4-7 of B, warp 8 TMA (ring of K and V tiles in the order of use),
// warps 9 and 10 the MMAs of A and of B.
// All waits are bounded.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "prompt_plan.h"
#include "tc_ptx.cuh"

namespace skv {

namespace {

constexpr int kTile = 128;
constexpr int kThreads = 384;         // three warpgroups; the last one's warp 3 idles
// Registers: 384 threads start with 168; the softmax warpgroups hold a whole row of scores, so they
// take 208 and the third gives up to 88 (2 x 128 x 208 + 128 x 88 = 384 x 168).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "the split fits the launch's registers");
constexpr int kRegion = kTile * 128;  // 16 KB: 128 rows of 64 bf16
constexpr float kRaise = 8.f;

template <int D>
struct Smem {
  static constexpr int tile = D / 64 * kRegion;
  static constexpr int slots = D == 128 ? 5 : 8;
  static constexpr int q = 0;                       // Q_A, Q_B
  static constexpr int kv = 2 * tile;
  static constexpr int bars = kv + slots * tile;
  static constexpr int nbars = 2 * slots + 2 + 8;
  static constexpr int misc = bars + nbars * 8;
  static constexpr int total = misc + 16;
};
static_assert(Smem<128>::total + 1024 <= 232448, "fits the 227 KB opt-in shared memory");

struct PromptArgs {
  const PromptItem* items;
  const int32_t* cta_indptr;
  int hq, group, total_q;
  float scale_log2;
  void* o;
  float* lse;
  float* o_part;
  float* lse_part;
  int32_t* status;
};

// D[tmem] (+)= A[tmem] . B[smem], kind::f16: A rows in TMEM lanes, two bf16 per column
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ uint64_t pk2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void upk2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// a += low half, b += high half, exact operands and one fp32 rounding each
__device__ __forceinline__ void add_bf16x2(float& a, float& b, uint32_t h) {
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tadd.rn.f32.bf16 %0, x, %0;\n\tadd.rn.f32.bf16 %1, y, %1;\n\t}"
      : "+f"(a), "+f"(b)
      : "r"(h));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// One row of a tile: p = 2^(s * scale - m), bf16 pairs into the row's P columns, the sum of the exact p
// into la and of the rounded ones into lb (as bf16 addends: 956 us on 4096 query tokens over 16384 keys, 32/8 heads;
// widened and added in pairs 970; without them 920, 16 ragged prompts 204, 222 and 196).
// (Two to four of every eight pairs by a polynomial on the FMA pipe measured slower: 1038 and 1118 us
// against 1011; the warps are bound by instructions, not by the exponential unit.)
__device__ __forceinline__ void weights(const float (&s)[kTile], uint64_t sc2, uint64_t nm2, uint32_t ts,
                                        uint64_t (&la)[2], float (&lb)[4]) {
#pragma unroll
  for (int c = 0; c < kTile; c += 32) {
    float pw[16];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const uint64_t x2 = fma2(pk2(s[c + e], s[c + e + 1]), sc2, nm2);
      float p0, p1;
      upk2(x2, p0, p1);
      p0 = ex2(p0);
      p1 = ex2(p1);
      const __nv_bfloat162 h2 = __floats2bfloat162_rn(p0, p1);
      const uint32_t h = *reinterpret_cast<const uint32_t*>(&h2);
      pw[e >> 1] = __uint_as_float(h);
      la[(e >> 1) & 1] = add2(la[(e >> 1) & 1], pk2(p0, p1));
      add_bf16x2(lb[e & 2], lb[(e & 2) + 1], h);
    }
    tc::tmem_st_x16(ts + c / 2, pw);
  }
}

// 32 bytes, one whole sector, in one store where the address allows it (`whole`)
__device__ __forceinline__ void store32(void* p, const uint32_t (&u)[8], bool whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                 "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    static_cast<uint4*>(p)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
}

// The two query tiles of an item, and the key tiles [0, tiles) of its range that each one needs.
struct Side {
  int q0, n, head, limit, tiles;
};
__device__ __forceinline__ Side side_of(const PromptItem& w, int x) {
  Side s;
  s.q0 = x ? w.q0b : w.q0a;
  s.n = x ? w.nb : w.na;
  s.head = x ? w.hb : w.ha;
  s.limit = x ? w.limit_b : w.limit_a;  // keys the tile's first token sees (all of them: not causal)
  const int64_t most = w.causal ? min((int64_t)w.kv_len, (int64_t)s.limit + s.n - 1) : (int64_t)w.kv_len;
  const int end = most > 0 ? (int)((most + kTile - 1) / kTile) : 0;
  s.tiles = s.n > 0 ? max(0, min(w.tile_end, end) - w.tile_begin) : 0;
  return s;
}

template <int D, typename OutT>
__global__ void __launch_bounds__(kThreads, 1)
prompt_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const PromptArgs a) {
  using S = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = tc::smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i_begin = a.cta_indptr[blockIdx.x], i_end = a.cta_indptr[blockIdx.x + 1];
  tc::grid_launch_dependents();  // the merge pass may be scheduled; it waits for this grid

  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + S::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::misc + 4);
  const uint32_t bar0 = sbase + S::bars;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S::slots + s); };
  const uint32_t qfull = bar0 + 8u * (2 * S::slots), qempty = qfull + 8;
  auto sfull_bar = [&](int x) { return qempty + 8u + 8u * x; };
  auto pfull_bar = [&](int x) { return qempty + 24u + 8u * x; };
  auto ofull_bar = [&](int x) { return qempty + 40u + 8u * x; };
  auto turn_bar = [&](int x) { return qempty + 56u + 8u * x; };

  if (tid == 0) {
    for (int s = 0; s < S::slots; ++s) {
      tc::mbar_init(full_bar(s), 1);
      tc::mbar_init(empty_bar(s), 2);  // both sides
    }
    tc::mbar_init(qfull, 1);
    tc::mbar_init(qempty, 2);
    for (int x = 0; x < 2; ++x) {
      tc::mbar_init(sfull_bar(x), 1);
      tc::mbar_init(pfull_bar(x), 4);
      tc::mbar_init(ofull_bar(x), 1);
      tc::mbar_init(turn_bar(x), 1);
    }
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 9) tc::tmem_alloc(tc::smem_u32(tmem_holder), 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t tm_s[2] = {tmem, tmem + kTile}, tm_o[2] = {tmem + 2 * kTile, tmem + 3 * kTile};

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ==================================================================================== TMA
      int slot_it = 0, q_it = 0;  // ring loads and Q loads so far
      bool ok = true;
      auto load_kv = [&](const CUtensorMap* map, int head, int row) {
        const int st = slot_it % S::slots;
        if (slot_it >= S::slots) ok = tc::mbar_wait(empty_bar(st), ((slot_it / S::slots) + 1) & 1, abort_flag, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(full_bar(st), (uint32_t)S::tile);
          for (int r = 0; r < D / 64; ++r)
            tc::tma_load_3d(sbase + S::kv + st * S::tile + r * kRegion, map, full_bar(st), r * 64, head, row);
        }
        ++slot_it;
      };
      if (lane == 0) {
        tc::prefetch_tmap(&qmap);
        tc::prefetch_tmap(&kmap);
        tc::prefetch_tmap(&vmap);
      }
      for (int i = i_begin; i < i_end && ok; ++i) {
        const PromptItem w = a.items[i];
        const Side sa = side_of(w, 0), sb = side_of(w, 1);
        const int tiles = max(sa.tiles, sb.tiles);
        if (tiles == 0) continue;
        if (q_it > 0) ok = tc::mbar_wait(qempty, (q_it + 1) & 1, abort_flag, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          const int sides = (sa.tiles > 0) + (sb.tiles > 0);
          tc::mbar_arrive_expect_tx(qfull, (uint32_t)(sides * S::tile));
          for (int r = 0; r < D / 64; ++r) {
            if (sa.tiles > 0) tc::tma_load_3d(sbase + S::q + r * kRegion, &qmap, qfull, r * 64, sa.head, sa.q0);
            if (sb.tiles > 0) tc::tma_load_3d(sbase + S::q + S::tile + r * kRegion, &qmap, qfull, r * 64, sb.head, sb.q0);
          }
        }
        ++q_it;
        const int kh = w.ha / a.group, row0 = w.kv0 + w.tile_begin * kTile;
        load_kv(&kmap, kh, row0);
        for (int j = 0; j < tiles && ok; ++j) {  // in the order of use
          load_kv(&vmap, kh, row0 + j * kTile);
          if (ok && j + 1 < tiles) load_kv(&kmap, kh, row0 + (j + 1) * kTile);
        }
      }
      if (!ok && lane == 0) {  // copies in flight may still be landing: wait for them (bounded)
        auto drain = [&](uint32_t bar, uint32_t parity) {
          const uint64_t t0 = tc::globaltimer_ns();
          while (!tc::mbar_try_wait(bar, parity) && tc::globaltimer_ns() - t0 < 20000000ull) {
          }
        };
        for (int t = max(0, slot_it - S::slots); t < slot_it; ++t) drain(full_bar(t % S::slots), (t / S::slots) & 1);
        if (q_it > 0) drain(qfull, (q_it - 1) & 1);
      }
    } else if (warp < 11) {
      // =================================================================== MMA of one query tile
      // The whole warp keeps the loop and the waits; lane 0 issues.  (A lane that waits alone, with the
      // others parked at the end of the kernel, wakes late: 976 us against 957 with whole-warp waits.)
      constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, kTile, false, false);
      constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, D, false, true);
      const int x = warp - 9;
      const uint32_t qs = sbase + S::q + x * S::tile, ts = tm_s[x], to = tm_o[x];
      int slot_it = 0, q_it = 0, p_it = 0, turn = 0;
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort_flag, a.status)) && ok;
      };
      // A and B issue in turns, one group (P V, then the next Q K^T) each
      auto take_turn = [&]() {
        if (x == 1) wait(turn_bar(1), turn & 1);
        else if (turn > 0) wait(turn_bar(0), (turn - 1) & 1);
        ++turn;
      };
      auto wait_slot = [&]() {
        const int st = slot_it % S::slots;
        wait(full_bar(st), (slot_it / S::slots) & 1);
        ++slot_it;
        return st;
      };
      // a tile or Q handed back: when the MMAs that read it are done, or at once where none did
      auto release = [&](uint32_t bar, bool used) {
        if (used) tc::mma_commit(bar);
        else tc::mbar_arrive(bar);
      };
      auto qk = [&](int st) {
        const uint32_t ks = sbase + S::kv + st * S::tile;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_bf16(ts, tc::sdesc_sw128(qs + (k >> 2) * kRegion + (k & 3) * 32, 16, 1024),
                       tc::sdesc_sw128(ks + (k >> 2) * kRegion + (k & 3) * 32, 16, 1024), idesc_s, k > 0 ? 1u : 0u);
        tc::mma_commit(sfull_bar(x));
      };
      for (int i = i_begin; i < i_end && ok; ++i) {
        const PromptItem w = a.items[i];
        const int tiles = side_of(w, x).tiles, all = max(tiles, side_of(w, 1 - x).tiles);
        if (all == 0) continue;
        wait(qfull, q_it & 1);
        ++q_it;
        int kst = wait_slot();
        take_turn();
        if (!ok) break;
        tc::tc_fence_after();
        if (lane == 0) {
          if (tiles > 0) qk(kst);
          tc::mbar_arrive(turn_bar(1 - x));
          release(empty_bar(kst), tiles > 0);
          if (tiles <= 1) release(qempty, tiles > 0);
        }
        __syncwarp();
        for (int j = 0; j < all; ++j) {
          const int vst = wait_slot();
          if (j + 1 < all) kst = wait_slot();
          take_turn();  // free long before P is: one wait less behind P
          if (j < tiles) {
            wait(pfull_bar(x), p_it & 1);
            ++p_it;
          }
          if (!ok) break;
          tc::tc_fence_after();
          if (lane == 0) {
            if (j < tiles) {
              const uint32_t vs = sbase + S::kv + vst * S::tile;
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k)  // 16 keys: 8 packed columns of P
                mma_ts(to, ts + k * 8, tc::sdesc_sw128(vs + k * 2048, kRegion, 1024), idesc_o,
                       (j > 0 || k > 0) ? 1u : 0u);
              if (j + 1 == tiles) tc::mma_commit(ofull_bar(x));
            }
            if (j + 1 < tiles) qk(kst);
            tc::mbar_arrive(turn_bar(1 - x));
            release(empty_bar(vst), j < tiles);
            if (j + 1 < all) release(empty_bar(kst), j + 1 < tiles);
            if (j + 2 == tiles) tc::mma_commit(qempty);
          }
          __syncwarp();
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ================================================================================ softmax
    const int x = warp >> 2, quarter = warp & 3;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tm_s[x] + lane_base, to = tm_o[x] + lane_base;
    const int r = quarter * 32 + lane;  // this thread's row of the tile
    int s_it = 0, o_it = 0;
    int v_seq = 0;  // ring loads of the items before this one
    bool ok = true;
    PromptItem next = a.items[i_begin];  // the planner leaves no CTA without an item
    for (int i = i_begin; i < i_end; ++i) {
      const PromptItem w = next;
      const Side s_me = side_of(w, x);
      const int tiles = s_me.tiles, all_tiles = max(tiles, side_of(w, 1 - x).tiles);
      // P V multiplies the weights rounded to bf16, each off by 2^-8 of itself at most (half a step, as a
      // bf16 O is from its own value).  l: sum of the exact weights, for the LSE; lr: of the rounded ones, O's divisor, so that keys
      // of one value return it, and a row dominated by one key that key's V, whatever the weights' rounding
      float m = -INFINITY, l = 0.f, lr = 0.f;
      const int64_t lim64 = w.causal ? min((int64_t)w.kv_len, (int64_t)s_me.limit + r) : (int64_t)w.kv_len;
      const int limit = (int)max(lim64, (int64_t)0);
      const int warp_limit = __shfl_sync(0xffffffffu, limit, 0);  // the warp's first row sees fewest
      for (int j = 0; j < tiles; ++j) {
        const int key0 = (w.tile_begin + j) * kTile;
        ok = tc::mbar_wait(sfull_bar(x), s_it & 1, abort_flag, a.status) && ok;
        ++s_it;
        tc::tc_fence_after();
        float s[kTile];
#pragma unroll
        for (int c = 0; c < kTile; c += 16) {
          float v[16];
          tc::tmem_ld_x16(ts + c, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) s[c + e] = v[e];
        }
        tc::tmem_wait_ld();
        if (key0 + kTile > warp_limit) {
          const int nv = limit - key0;
#pragma unroll
          for (int c = 0; c < kTile; ++c) s[c] = c < nv ? s[c] : -INFINITY;
        }
        float mx;
        {
          float q[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            q[u] = max3(s[32 * u], s[32 * u + 1], s[32 * u + 2]);
#pragma unroll
            for (int e = 3; e < 31; e += 2) q[u] = max3(q[u], s[32 * u + e], s[32 * u + e + 1]);
            q[u] = fmaxf(q[u], s[32 * u + 31]);
          }
          mx = fmaxf(fmaxf(q[0], q[1]), fmaxf(q[2], q[3])) * a.scale_log2;  // the scale is positive
        }
        const bool raise = mx > m + kRaise;
        if (__any_sync(0xffffffffu, raise)) {  // warp-uniform: TMEM access is warp-collective
          const float mn = raise ? mx : m;
          const float al = mn == m ? 1.f : ex2(m - mn);
          l *= al;
          lr *= al;
          m = mn;
          if (j > 0) {  // a full S(j) means P V(j - 1) is done
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float v[16];
              tc::tmem_ld_x16(to + c, v);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] *= al;
              tc::tmem_st_x16(to + c, v);
            }
          }
        }
        if (key0 + kTile > w.kv_len) {
          // keys past the sequence belong to another one (or to nobody): their V rows become zero
          // before either side multiplies them (both sides may write the same zeros)
          const int seq = v_seq + 2 * j + 1;  // ring position of V(j)
          const int st = seq % S::slots;
          ok = tc::mbar_wait(full_bar(st), (seq / S::slots) & 1, abort_flag, a.status) && ok;
          uint8_t* vb = smem + S::kv + st * S::tile;
          if (r >= w.kv_len - key0) {
#pragma unroll
            for (int rgn = 0; rgn < D / 64; ++rgn)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                reinterpret_cast<uint4*>(vb + rgn * kRegion + r * 128)[e] = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async_smem();
        }
        const float mm = m == -INFINITY ? 0.f : m;
        const uint64_t sc2 = pk2(a.scale_log2, a.scale_log2), nm2 = pk2(-mm, -mm);
        uint64_t la[2] = {0, 0};
        float lb[4] = {0.f, 0.f, 0.f, 0.f};
        weights(s, sc2, nm2, ts, la, lb);
        {
          float a0, a1;
          upk2(add2(la[0], la[1]), a0, a1);
          l += a0 + a1;
          lr += (lb[0] + lb[1]) + (lb[2] + lb[3]);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(pfull_bar(x));
      }
      v_seq += 2 * all_tiles;
      if (tiles > 0) {
        ok = tc::mbar_wait(ofull_bar(x), o_it & 1, abort_flag, a.status) && ok;
        ++o_it;
        tc::tc_fence_after();
      }
      next = a.items[min(i + 1, i_end - 1)];  // on its way while the results are stored
      const bool some = l > 0.f || l != l;
      const float inv = some ? 1.f / lr : 0.f;
      const int rows = min(s_me.n, a.total_q - s_me.q0);
      const bool part = w.part_row >= 0;
      // this tile's first row, and rows a token apart
      const int64_t row0 = part ? (int64_t)w.part_row + (int64_t)(s_me.q0 - w.q0a) * w.part_stride : (int64_t)s_me.q0;
      const int64_t step = part ? w.part_stride : 1;
      float* const lse = part ? a.lse_part : a.lse;
      if (r < rows && lse != nullptr)
        lse[(row0 + r * step) * a.hq + s_me.head] = some ? (m + log2f(l)) * kLn2 : -INFINITY;
      const bool fp32 = part || sizeof(OutT) == 4;
      const int64_t out = ((row0 + r * step) * a.hq + s_me.head) * D;
      uint8_t* dst = part ? reinterpret_cast<uint8_t*>(a.o_part + out)
                          : reinterpret_cast<uint8_t*>(reinterpret_cast<OutT*>(a.o) + out);
      const bool whole = (reinterpret_cast<uintptr_t>(part ? a.o_part : a.o) & 31) == 0;  // rows are whole sectors
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        float v[16];
        if (tiles > 0) {  // the whole warp loads; live rows store
          tc::tmem_ld_x16(to + c, v);
          tc::tmem_wait_ld();
        }
        uint32_t u[8], u2[8];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = some ? v[e] * inv : 0.f;
        if (fp32) {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(v[e]), u2[e] = __float_as_uint(v[8 + e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
            u[e] = *reinterpret_cast<const uint32_t*>(&h2);
          }
        }
        if (r < rows) {
          store32(dst, u, whole);
          if (fp32) store32(dst + 32, u2, whole);
        }
        dst += fp32 ? 64 : 32;
      }
      tc::tc_fence_before();  // O has been read before the next item's first P is announced
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
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

// [rows, heads, D] bf16 with (row, head) strides in elements; 128-row boxes of one head's 64 columns.
bool rows_map(CUtensorMap* m, const void* base, int rows, int heads, int head_dim, const int64_t* stride) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  // the stride of a dimension of one entry is never used, but has to be a valid one
  const cuuint64_t head_st = heads > 1 ? (cuuint64_t)stride[1] * 2 : (cuuint64_t)head_dim * 2;
  const cuuint64_t row_st = rows > 1 ? (cuuint64_t)stride[0] * 2 : (cuuint64_t)head_dim * 2 * heads;
  const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t st[2] = {head_st, row_st};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)kTile}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, st, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, typename OutT>
int launch_t(const CUtensorMap* maps, const PromptArgs& a, int ctas, cudaStream_t s) {
  static DeviceSmemAttr attr;
  const int smem = Smem<D>::total + 1024;
  if (const int e = attr.ensure(reinterpret_cast<const void*>(prompt_attn_kernel<D, OutT>), smem)) return e;
  prompt_attn_kernel<D, OutT><<<ctas, kThreads, smem, s>>>(maps[0], maps[1], maps[2], a);
  return (int)cudaGetLastError();
}

}  // namespace

int launch_prompt_attn(const skv_prompt_params& p, const PromptItem* items, const int32_t* cta_indptr, int num_ctas,
                       cudaStream_t s) {
  CUtensorMap maps[3];
  if (!rows_map(&maps[0], p.q, p.total_q, p.num_qo_heads, p.head_dim, p.q_stride)) return (int)cudaErrorInvalidValue;
  if (p.total_kv > 0) {
    if (!rows_map(&maps[1], p.k, p.total_kv, p.num_kv_heads, p.head_dim, p.k_stride) ||
        !rows_map(&maps[2], p.v, p.total_kv, p.num_kv_heads, p.head_dim, p.v_stride))
      return (int)cudaErrorInvalidValue;
  } else {  // no key anywhere: the maps are never used
    maps[1] = maps[0];
    maps[2] = maps[0];
  }
  PromptArgs a;
  a.items = items;
  a.cta_indptr = cta_indptr;
  a.hq = p.num_qo_heads;
  a.group = p.num_qo_heads / p.num_kv_heads;
  a.total_q = p.total_q;
  a.scale_log2 = p.sm_scale * kLog2e;
  a.o = p.o;
  a.lse = p.lse;
  a.o_part = p.o_part;
  a.lse_part = p.lse_part;
  a.status = p.status;
  const bool bf16 = p.o_dtype == SKV_BF16;
  if (p.head_dim == 128)
    return bf16 ? launch_t<128, __nv_bfloat16>(maps, a, num_ctas, s) : launch_t<128, float>(maps, a, num_ctas, s);
  return bf16 ? launch_t<64, __nv_bfloat16>(maps, a, num_ctas, s) : launch_t<64, float>(maps, a, num_ctas, s);
}

}  // namespace skv
