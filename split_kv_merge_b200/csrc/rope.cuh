// Rotary positions on rows of heads: the angle arithmetic, the (cos, sin) table of a few tokens in
// shared memory, and 16-value pieces of a row as they are loaded, turned and stored.
#pragma once
#include <math.h>
#include <string.h>

#include "skv_common.cuh"

namespace skv {
namespace rope {

constexpr int kMaxDim = 256;
constexpr int kMaxPairs = kMaxDim / 2;

// Frequencies of a launch in 2^-64 turns per position.  position * turns[p] in wrapping 64-bit
// arithmetic is the angle's fraction of a turn, with no range reduction to lose bits in: the error
// is position * 2^-64 turns (2^-33 at position 2^31), below fp32's own rounding of the result.
struct Freq {
  uint64_t turns[kMaxPairs];
  float mscale;
  int dim, halves;
};

// Host: w radians in 2^-64 turns, nearest below, whole turns dropped (positions are integers).
// |w| < 2^32.  Integer product of w's 53-bit mantissa with 1 / (2 pi) held to 128 bits.
inline uint64_t to_turns(double w) {
  uint64_t bits;
  memcpy(&bits, &w, 8);
  const int e = (int)(bits >> 52) & 0x7FF;             // |w| = mant 2^(e - 1075)
  const uint64_t mant = (bits & ((1ull << 52) - 1)) | (e > 0 ? 1ull << 52 : 0);
  const unsigned __int128 hi = (unsigned __int128)mant * 0x28BE60DB9391054Aull;
  const unsigned __int128 lo = (unsigned __int128)mant * 0x7F09D5F47D4D3770ull;
  const unsigned __int128 p = hi + (lo >> 64);         // 2^-64 turns before the factor 2^(e - 1075)
  const int down = 1075 - (e > 0 ? e : 1);             // > 20
  const uint64_t t = down > 127 ? 0 : (uint64_t)(p >> down);
  return (bits >> 63) ? (uint64_t)0 - t : t;
}

// Host: the table of an skv_rope (validated by the caller), negated for the inverse rotation.
inline void make_freq(const skv_rope& r, bool inverse, Freq* f) {
  for (int p = 0; p < r.dim / 2; ++p) {
    const double w = r.inv_freq_h != nullptr ? r.inv_freq_h[p] : pow(r.theta, -2.0 * p / r.dim);
    f->turns[p] = to_turns(inverse ? -w : w);
  }
  f->mscale = r.mscale;
  f->dim = r.dim;
  f->halves = r.layout == SKV_ROPE_HALVES;
}

// Host: tokens a block of threads takes when a token has `work` items: two items a thread at least, and
// so many blocks (32 an SM) that their last wave is a small part of the run.
inline int tokens_per_block(int64_t tokens, int work, int threads, int most, int64_t sms) {
  const int64_t fill = (2 * threads + work - 1) / work, share = tokens / (sms * 32);
  const int64_t n = fill > share ? fill : share;
  return (int)(n < 1 ? 1 : n > most ? most : n);
}

// (cos, sin) of pos * turns * 2^-64 of a turn, times mscale.  The nearest quarter turn comes off in
// integers, so the fp32 angle that is left lies within +-1/8 turn and keeps 2^-32 of a turn.  There,
// with y in half turns and z = y^2, sin = y (S0 + S1 z + S2 z^2 + S3 z^3) and cos = 1 + z (C1 + ..), least
// maximum error fits: 2.1 x 2^-24 of the sine, 0.9 x 2^-24 for the cosine when evaluated in fp32.
__device__ __forceinline__ float2 cos_sin(int32_t pos, uint64_t turns, float mscale) {
  const uint64_t u = (uint64_t)(int64_t)pos * turns + (1ull << 61);
  const uint32_t hi = (uint32_t)(u >> 32), quad = hi >> 30;
  const int32_t rem = (int32_t)(((uint32_t)(u >> 30)) - 0x80000000u);  // 2^-34 turns, [-2^31, 2^31)
  const float y = (float)rem * 1.16415321826934814453125e-10f;         // 2^-33: half turns, |y| <= 1/4
  const float z = y * y;
  float s = fmaf(z, -0.5890122056f, 2.5497610569f), c = fmaf(z, 0.2314295471f, -1.3350584507f);
  s = fmaf(z, s, -5.1677079201f);
  c = fmaf(z, c, 4.0587077141f);
  s = fmaf(z, s, 3.1415927410f);
  c = fmaf(z, c, -4.9348020554f);
  s *= y;
  c = fmaf(z, c, 1.f);
  const float cc = (quad & 1) ? s : c, ss = (quad & 1) ? c : s;
  return make_float2(((quad == 1 || quad == 2) ? -cc : cc) * mscale, ((quad & 2) ? -ss : ss) * mscale);
}

// A row of D values is cut into items of 16, two chunks of 8 half a part of the row apart, so that the
// lanes of a row read and write consecutive chunks (with 16 consecutive values a lane, each 32-byte
// sector was written by two instructions).  Item i < dim/16 holds chunks i and dim/16 + i and
// with them eight whole pairs: (x[p], x[8+p]) for halves, (x[2p], x[2p+1]) for interleaved pairs, four in
// each chunk.  Later items are copied.  The table of a token holds item i's pairs (2j, 2j+1) as one
// float4 at [j][i], so the lanes of a row read consecutive 16-byte words.
__device__ __forceinline__ int table_float4s(int dim) { return dim / 4; }

// Block-wide: the frequencies into shared memory.  (Lanes that index the parameter bank apart are served
// one after another; once a block that is bearable, once a table entry it is not.)
__device__ __forceinline__ void stage_turns(uint64_t* turns, const Freq& f, int tid, int threads) {
  for (int p = tid; p < f.dim / 2; p += threads) turns[p] = f.turns[p];
}

// Block-wide: the table of `n` tokens whose positions are pos[0..n).
__device__ __forceinline__ void fill_table(float4* table, const int32_t* pos, int n, const uint64_t* turns, int dim,
                                           float mscale, bool halves, int tid, int threads) {
  const int half = dim / 2, items = dim / 16;
  if (half == 0) return;  // nothing turns
  float2* t2 = reinterpret_cast<float2*>(table);
  int tok = tid / half, p = tid - tok * half;  // then on by `threads` pairs, without dividing again
  const int tok_step = threads / half, p_step = threads - tok_step * half;
  while (tok < n) {
    // halves: pair p is number p % 8 of item p / 8; interleaved: of chunk p / 4, which is the item's first or
    // second one
    const int second = !halves && p >= 4 * items, i = halves ? p >> 3 : (p >> 2) - (second ? items : 0);
    const int j = halves ? (p & 7) >> 1 : 2 * second + ((p & 3) >> 1);
    t2[tok * half + (j * items + i) * 2 + (p & 1)] = cos_sin(pos[tok], turns[p], mscale);
    tok += tok_step;
    p += p_step;
    if (p >= half) {
      p -= half;
      ++tok;
    }
  }
}

// Element offsets of an item's two chunks.
struct Item {
  int c0, c1;
  bool turned, two;
};
__device__ __forceinline__ Item item_of(int i, int dim, int head_dim) {
  Item it;
  const int nrot = dim / 16, rest = ((head_dim - dim) / 8 + 1) / 2;  // items turned and copied
  it.turned = i < nrot;
  it.c0 = it.turned ? i * 8 : dim + (i - nrot) * 8;
  it.c1 = it.c0 + (it.turned ? nrot : rest) * 8;
  it.two = it.c1 < head_dim;
  return it;
}

// x holds the 16 values in chunk order; turned by the token's table entries of item i.
__device__ __forceinline__ void turn_item(float (&x)[16], const float4* tok_table, int i, int items, bool halves) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 cs = tok_table[j * items + i];
    // pairs 2j and 2j+1 of the item: (x[p], x[8+p]) for halves, (x[2p], x[2p+1]) interleaved
    if (halves) {
      const float a0 = x[2 * j], b0 = x[8 + 2 * j], a1 = x[2 * j + 1], b1 = x[9 + 2 * j];
      x[2 * j] = a0 * cs.x - b0 * cs.y;
      x[8 + 2 * j] = a0 * cs.y + b0 * cs.x;
      x[2 * j + 1] = a1 * cs.z - b1 * cs.w;
      x[9 + 2 * j] = a1 * cs.w + b1 * cs.z;
    } else {
      const float a0 = x[4 * j], b0 = x[4 * j + 1], a1 = x[4 * j + 2], b1 = x[4 * j + 3];
      x[4 * j] = a0 * cs.x - b0 * cs.y;
      x[4 * j + 1] = a0 * cs.y + b0 * cs.x;
      x[4 * j + 2] = a1 * cs.z - b1 * cs.w;
      x[4 * j + 3] = a1 * cs.w + b1 * cs.z;
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x);
  x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z);
  x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// One item's raw words of a row, so that loads can be issued ahead of their use.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* row, const Item& it) {
    a = *reinterpret_cast<const uint4*>(row + it.c0);
    b = it.two ? *reinterpret_cast<const uint4*>(row + it.c1) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void values(float (&x)[16]) const {
    unpack8(a, x);
    unpack8(b, x + 8);
  }
};
template <>
struct Raw<float> {
  float4 a, b, c, d;
  __device__ __forceinline__ void load(const float* row, const Item& it) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    a = *reinterpret_cast<const float4*>(row + it.c0);
    b = *reinterpret_cast<const float4*>(row + it.c0 + 4);
    c = it.two ? *reinterpret_cast<const float4*>(row + it.c1) : z;
    d = it.two ? *reinterpret_cast<const float4*>(row + it.c1 + 4) : z;
  }
  __device__ __forceinline__ void values(float (&x)[16]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    x[8] = c.x; x[9] = c.y; x[10] = c.z; x[11] = c.w;
    x[12] = d.x; x[13] = d.y; x[14] = d.z; x[15] = d.w;
  }
};
__device__ __forceinline__ void store_item(__nv_bfloat16* row, const Item& it, const float (&x)[16]) {
  *reinterpret_cast<uint4*>(row + it.c0) = pack8(x);
  if (it.two) *reinterpret_cast<uint4*>(row + it.c1) = pack8(x + 8);
}
__device__ __forceinline__ void store_item(float* row, const Item& it, const float (&x)[16]) {
  *reinterpret_cast<float4*>(row + it.c0) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(row + it.c0 + 4) = make_float4(x[4], x[5], x[6], x[7]);
  if (it.two) {
    *reinterpret_cast<float4*>(row + it.c1) = make_float4(x[8], x[9], x[10], x[11]);
    *reinterpret_cast<float4*>(row + it.c1 + 4) = make_float4(x[12], x[13], x[14], x[15]);
  }
}

}  // namespace rope
}  // namespace skv
