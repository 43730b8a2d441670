// The cache of a draft held in 4 bits: its writing, its reading back, and the
// attention of a round's positions over it, with a sliding window and sinks.
//
// A token's key (and value) of one head is D codes c of 4 bits with a bf16 scale s
// and a bf16 minimum m, value m + s c.  A page holds, head by head, the codes of
// its tokens' keys, then of their values (D / 2 bytes each, the even value in a
// byte's low half), then four bytes (s, m) for each key and for each value.
//
// Attention lays the key tiles (16 tokens) of all (sequence, key head, block of query rows)
// groups in a row and gives every warp that the card holds an even share of it, whatever the
// lengths are: a share begins and ends inside a group.  A warp works alone, with a softmax state
// of its own; the warp that is the last to finish a cut group joins its parts, in the order of
// the tokens.  (With four warps of a CTA to a group, barriers between them and a copy per 16
// bytes the 256 sequences below took 178 us, with warps by themselves and bulk copies 152.)
//   z_j = scale (s_j q.c_j + m_j sum q)      S^T = C_K Q^T, 16 tokens by 8 rows
//   o   = sum_j p_j m'_j + sum_j (p_j s'_j) c'_j       O^T = C_V^T P^T
// so that the tensor cores see the codes themselves and the scales stay in float32.  With the
// tokens on the 16-row side of mma.m16n8k16 a step of one query position (8 rows of a key
// head) wastes nothing, and codes never leave registers: 4 bits at the bottom of a half are
// the fp16 subnormal c 2^-24 (8 bits up c 2^-20), exact, so one AND makes two operands.  Q is
// fp16 with a power of two per row, which keeps bf16's 8 bits down to 2^-27 of the row's
// largest value; p_j s'_j is fp16 next to a running maximum of its own (2^7 to 2^15 there, so that the maximum may
// grow by 2^8 before sums are scaled: 11 bits down to 2^-21 of the largest, 2^-32 of it below; the plain float32
// form's distance from 64 bits is the output's own rounding, 0.0017, and so is this one's).
//
// 256 sequences of up to 4096 tokens, 32 query and 8 key heads of 128: 122 us, 592 MB at 72% of
// the measured copy rate, and next to that bound by the integer instructions that take codes
// apart (half the rate of the others; 53% of the slots).  64 sequences, 1 to 4 positions, a window
// of 1024: 35 us for 75 MB, some 15 of it the way to the first tile and the joins of the parts.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "sv_kv4_shares.h"
#include "sv_tc.cuh"

namespace sv {
namespace kv4 {

// Quotient of 0 <= n < 2^31 by a fixed divisor: n * ceil(2^(31 + l) / d) / 2^(31 + l) with
// l = ceil(log2 d) (its error, below 2^l n / 2^(31 + l) < 1 steps of 1/d, never reaches the next).
struct Divider {
  uint32_t magic, shift, one;
};
inline Divider divider(int d) {
  int l = 0;
  while ((1LL << l) < d) ++l;
  if (l == 0) return {0, 0, 1};
  const unsigned long long p = 1ull << (31 + l);
  return {(uint32_t)((p + d - 1) / d), (uint32_t)(l - 1), 0};
}
__device__ __forceinline__ int divide(int n, const Divider& d) {
  return d.one ? n : (int)(__umulhi((uint32_t)n, d.magic) >> d.shift);
}

struct Cache {
  uint8_t* pool;
  long long page_bytes;
  int head_bytes, num_pages, page_size, max_pages;
  Divider by_page;
  const int32_t* table;
};

inline Cache cache_of(const Kv4Cache& c, int D) {
  Cache r;
  r.pool = static_cast<uint8_t*>(c.pool);
  r.head_bytes = (int)kv4_head_bytes(D, c.page_size);
  r.page_bytes = (long long)r.head_bytes * c.Hkv;
  r.num_pages = c.num_pages;
  r.page_size = c.page_size;
  r.max_pages = c.max_pages;
  r.by_page = divider(c.page_size);
  r.table = c.table;
  return r;
}

// ---------------------------------------------------------------------------
// Writing and reading.  D / 16 lanes share a row, 16 values of it each: two words of codes.  A CTA takes a
// few tokens of one sequence, kRowsAhead rows a thread, whose loads are all on their way before the first is
// used.  8 prompts of up to 4096 tokens and 8 heads: writing 42 us, reading back 28 us, where the bytes take
// 14 each; the instructions for addresses and codes bound both (73% and 68% of the issue slots).
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;
constexpr int kRowsAhead = 2;

struct RowArgs {
  Cache c;
  const int32_t* starts;
  const int32_t* n_per_row;
  const uint16_t* in[2];  // K, V
  void* out[2];
  long long seq, pos, head;  // elements
  int out_f32, B, T, Hkv, tokens;  // tokens of a CTA's turn
  Divider by_rows;           // 2 * Hkv, a token's
  uint32_t* flags;
};

// A sequence's tokens: n of them from `start`; 0 of one that is left out.
struct RowSeq {
  int b, n, start;
  const int32_t* table;
};
__device__ __forceinline__ RowSeq row_seq(const RowArgs& a, int b) {
  RowSeq q;
  q.b = b;
  q.n = a.n_per_row ? a.n_per_row[b] : a.T;
  q.start = a.starts[b];
  q.table = a.c.table + (long long)b * a.c.max_pages;
  if (q.n < 0 || q.n > a.T || q.start < 0 || (long long)q.start + q.n > (long long)a.c.max_pages * a.c.page_size) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(a.flags, SV_FLAG_BAD_N);
    q.n = 0;
  }
  return q;
}

// A thread's row: of token i, part 0 (K) or 1 (V), head h; its bytes in the pool.  One that is behind the last token or
// on a bad page is not `there`, and stands for another, so that nothing waits before its loads.
struct Row {
  int i, part, h;
  bool there;
  uint8_t* codes;
  int scale;  // from its codes to its (s, m)
};
template <int D>
__device__ __forceinline__ Row row_of(const RowArgs& a, const RowSeq& q, int first, int last, int r) {
  Row w;
  const int tok = divide(r, a.by_rows), rest = r - tok * 2 * a.Hkv;
  w.i = min(first + tok, last - 1);
  w.part = rest >= a.Hkv;
  w.h = rest - w.part * a.Hkv;
  const int t = q.start + w.i, p = divide(t, a.c.by_page), slot = t - p * a.c.page_size;
  const int page = q.table[p];
  const bool good = (unsigned)page < (unsigned)a.c.num_pages;
  if (!good && rest == 0) atomicOr(a.flags, SV_FLAG_BAD_PAGE);
  w.there = good && first + tok < last;
  const int half = a.c.page_size * (D / 2);  // (a page has fewer than 2^31 bytes)
  w.codes = a.c.pool + (unsigned long long)(good ? (uint32_t)page : 0u) * (uint32_t)a.c.page_bytes +
            (uint32_t)(w.h * a.c.head_bytes + w.part * half + slot * (D / 2));
  w.scale = (2 - w.part) * half + w.part * a.c.page_size * 4 - slot * (D / 2 - 4);
  return w;
}

// The smaller (larger) of two pairs of bf16; NaN if one is.
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Whether a row's x - m (m + s c) may have more than float32's 24 bits next to a border of its rounding: a minimum
// that is not 0, with an exponent below the scale's by more than 12.  A border is a multiple of s / 2 of at most
// 15.5 s (of bf16: at most 15 s + m), and x (s c) has 8 (12) bits, so otherwise every bit of m lies within the 24.
__device__ __forceinline__ bool far_apart(uint32_t s, uint32_t m) {  // bits of bf16
  return (int)(s >> 7 & 255u) - (int)(m >> 7 & 255u) > 12 && (m & 0x7fffu) != 0;
}

// What a row's codes take: minimum m and scale s > 0, by halves, since x - m may leave float32's range.
struct Coder {
  // half of x's factor, -m / 2, 2 / s, -s / 2; times 2^80 for a scale whose reciprocal may be infinite
  F2 hx, hm, inv, step;
  float half, below;     // half a step (of s / 2), and the value below

  __device__ __forceinline__ Coder(float m, float s) {
    const float up = s < 0x1p-60f ? 0x1p80f : 1.f;
    const float hs = 0.5f * s * up, x = 0.5f * up, y = -0.5f * m * up, r = __frcp_rn(hs);
    hx = f2_pack(x, x), hm = f2_pack(y, y), inv = f2_pack(r, r), step = f2_pack(-hs, -hs);
    half = 0.5f * hs;
    below = __uint_as_float(__float_as_uint(half) - 1u);
  }
  // Whether 0 - m lies on a border (an odd number of half steps), and one of 16 values is next to it: not 0, but 2^16 or
  // more times smaller than m.  Then x - m may be rounded onto that border.  (Another border is too far from m for an x
  // of so few bits, where the row is not far_apart.)
  __device__ __forceinline__ bool next_to_border(const uint4& v, const uint4& w, uint32_t m_bits) const {
    float low, r, same;
    f2_unpack(hm, low, same);
    f2_unpack(inv, r, same);
    const float y = __fmaf_rn(low, 2.f * r, 12582912.f);  // (-m in half steps)
    if (!(__float_as_uint(y) & 1u) || (y - 12582912.f) * half != low) return false;
    const uint32_t words[8] = {v.x, v.y, v.z, v.w, w.x, w.y, w.z, w.w};
    uint32_t least = ~0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) least = __vminu2(least, __vsub2(words[i] & 0x7fff7fffu, 0x00010001u));
    return (int)min(least & 0xffffu, least >> 16) < (int)(m_bits & 0x7fffu) - (16 << 7);
  }
  // Codes of 8 values: the nearest integers to (x - m) / s, ties to even.  The product with the reciprocal,
  // rounded by the addition of 1.5 2^23, is one off at most, where the quotient lies next to a border: the
  // remainder (exact: c and s have 4 and 8 bits) is then beyond half a step, or is half a step and c is odd.
  // Remainders of half a step or more are looked for together (of 8 normal values one in sixty has any).
  __device__ __forceinline__ uint32_t word(const uint4& v) const {
    const uint32_t pairs[4] = {v.x, v.y, v.z, v.w};
    const F2 magic = f2_pack(12582912.f, 12582912.f), less = f2_pack(-12582912.f, -12582912.f);
    float y[8], r[8], far = 0.f;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const F2 t = f2_fma(f2_pack(bf16_lo(pairs[p]), bf16_hi(pairs[p])), hx, hm);
      f2_unpack(f2_fma(t, inv, magic), y[2 * p], y[2 * p + 1]);
#pragma unroll
      for (int e = 2 * p; e < 2 * p + 2; ++e) y[e] = fminf(y[e], 12582927.f);  // (a subnormal scale may be rounded far down)
      f2_unpack(f2_fma(f2_add(f2_pack(y[2 * p], y[2 * p + 1]), less), step, t), r[2 * p], r[2 * p + 1]);
      far = fmaxf(far, fmaxf(fabsf(r[2 * p]), fabsf(r[2 * p + 1])));
    }
    if (far >= half) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (fabsf(r[e]) > (__float_as_uint(y[e]) & 1u ? below : half))
          y[e] = fminf(y[e] + (r[e] > 0.f ? 1.f : -1.f), 12582927.f);
    }
    // the codes are the low bits of their floats, and the rest of these is known
    uint32_t w = 0;
#pragma unroll
    for (int e = 7; e >= 0; --e) w = w * 16u + __float_as_uint(y[e]);
    return w - 0x4b400000u * 0x11111111u;
  }
};

// The same for a row that is far_apart, or a value next_to_border: x - m may have been rounded onto a border from
// either side, and what that rounding lost decides.  (In the function above it costs registers that every row pays
// for: the prompts take 50 us instead of 44.)
__device__ __noinline__ uint32_t far_word(uint4 v, float m, float s) {
  const uint32_t pairs[4] = {v.x, v.y, v.z, v.w};
  const float up = s < 0x1p-60f ? 0x1p80f : 1.f;
  const float hs = 0.5f * s * up, half = 0.5f * hs, low = -0.5f * m * up, r = __frcp_rn(hs);
  uint32_t w = 0;
  for (int e = 7; e >= 0; --e) {
    float t, lost;
    two_sum((e & 1 ? bf16_hi(pairs[e / 2]) : bf16_lo(pairs[e / 2])) * (0.5f * up), low, t, lost);
    float c = fminf(rintf(t * r), 15.f);
    const float rest = __fmaf_rn(-c, hs, t), beyond = rest < 0.f ? -lost : lost;
    const bool next = fabsf(rest) > half ||
                      (fabsf(rest) == half && (beyond > 0.f || (beyond == 0.f && ((int)c & 1))));
    if (next) c = fminf(c + (rest > 0.f ? 1.f : -1.f), 15.f);
    w = w << 4 | (uint32_t)c;
  }
  return w;
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) append_kernel(const __grid_constant__ RowArgs a) {
  constexpr int LANES = D / 16, PASS = kRowThreads / LANES, U = kRowsAhead;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % LANES, mine = threadIdx.x / LANES;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const RowSeq q = row_seq(a, b);
    for (long long at = (long long)blockIdx.x * a.tokens; at < q.n; at += (long long)gridDim.x * a.tokens) {
      const int first = (int)at, last = min(first + a.tokens, q.n), rows = (last - first) * 2 * a.Hkv;
      for (int r0 = 0; r0 < rows; r0 += U * PASS) {  // (every lane of a warp takes every turn)
        Row w[U];
        uint4 v[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          w[u] = row_of<D>(a, q, first, last, r0 + u * PASS + mine);
          const uint4* from = reinterpret_cast<const uint4*>((w[u].part ? a.in[1] : a.in[0]) + b * a.seq + w[u].i * a.pos +
                                                             w[u].h * a.head + lane * 16);
          v[u][0] = __ldcs(from);
          v[u][1] = __ldcs(from + 1);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t lo2 = min2(min2(v[u][0].x, v[u][0].y), min2(v[u][0].z, v[u][0].w));
          uint32_t hi2 = max2(max2(v[u][0].x, v[u][0].y), max2(v[u][0].z, v[u][0].w));
          lo2 = min2(lo2, min2(min2(v[u][1].x, v[u][1].y), min2(v[u][1].z, v[u][1].w)));
          hi2 = max2(hi2, max2(max2(v[u][1].x, v[u][1].y), max2(v[u][1].z, v[u][1].w)));
          lo2 = min2(lo2, lo2 >> 16 | lo2 << 16);
          hi2 = max2(hi2, hi2 >> 16 | hi2 << 16);
          uint32_t both = __byte_perm(lo2, hi2, 0x5410);  // the minimum and the maximum
#pragma unroll
          for (int m = 1; m < LANES; m <<= 1) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, both, m);
            both = __byte_perm(min2(both, o), max2(both, o), 0x7610);
          }
          if (!w[u].there) continue;
          const float lo = bf16_lo(both), hi = bf16_hi(both);
          // (max - min) / 15, correctly rounded twice: a float32 quotient of values with 8 bits lies on
          // a border of bf16 only if the exact one does
          const float s = 2.f * __fdiv_rn(0.5f * hi - 0.5f * lo, 15.f);
          uint16_t sb = __bfloat16_as_ushort(__float2bfloat16_rn(s)), mb = (uint16_t)both;
          const float sr = __uint_as_float((uint32_t)sb << 16);
          uint2 words = make_uint2(0, 0);
          if (!(isfinite(lo) && isfinite(hi))) {
            sb = mb = 0x7fc0u;  // a token that is not finite makes the scores of the queries that see it NaN
          } else if (sr > 0.f) {
            const Coder coder(lo, sr);
            if (far_apart(sb, mb) || coder.next_to_border(v[u][0], v[u][1], mb)) {
              words.x = far_word(v[u][0], lo, sr);
              words.y = far_word(v[u][1], lo, sr);
            } else {
              words.x = coder.word(v[u][0]);
              words.y = coder.word(v[u][1]);
            }
          }
          reinterpret_cast<uint2*>(w[u].codes)[lane] = words;
          if (lane == 0) *reinterpret_cast<uint32_t*>(w[u].codes + w[u].scale) = (uint32_t)sb | (uint32_t)mb << 16;
        }
      }
    }
  }
}

// The bf16 values of a word of codes of a row that is far_apart: to odd in float32, so that the rounding to bf16 is
// that of the value itself (to the nearest, a minimum below float32's bits may leave a border that the value is not on).
__device__ __noinline__ uint4 far_values(uint32_t word, float s, float m) {
  uint32_t v[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    float y[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float c = (float)(word >> (8 * p + 4 * e) & 15u), down = __fmaf_rd(c, s, m), up = __fmaf_ru(c, s, m);
      y[e] = __float_as_uint(down) & 1u ? down : up;
    }
    v[p] = tc::pack_bf16x2(y[0], y[1]);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const __grid_constant__ RowArgs a) {
  constexpr int LANES = D / 16, PASS = kRowThreads / LANES, U = kRowsAhead;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % LANES, mine = threadIdx.x / LANES;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const RowSeq q = row_seq(a, b);
    for (long long at = (long long)blockIdx.x * a.tokens; at < q.n; at += (long long)gridDim.x * a.tokens) {
      const int first = (int)at, last = min(first + a.tokens, q.n), rows = (last - first) * 2 * a.Hkv;
      for (int r0 = mine; r0 < rows; r0 += U * PASS) {
        Row w[U];
        uint2 words[U];
        uint32_t sm[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          w[u] = row_of<D>(a, q, first, last, r0 + u * PASS);
          words[u] = __ldcs(reinterpret_cast<const uint2*>(w[u].codes) + lane);
          sm[u] = *reinterpret_cast<const uint32_t*>(w[u].codes + w[u].scale);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (!w[u].there) continue;
          const float s = bf16_lo(sm[u]), m = bf16_hi(sm[u]);
          const F2 ss = f2_pack(s, s), mm = f2_pack(m, m), less = f2_pack(-8388608.f, -8388608.f);
          float y[16];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {  // (the codes as the low bits of 2^23 + c)
            const uint32_t word = e < 8 ? words[u].x : words[u].y;
            const uint32_t c0 = (word >> (4 * (e & 7)) & 15u) | 0x4b000000u;
            const uint32_t c1 = (word >> (4 * (e & 7) + 4) & 15u) | 0x4b000000u;
            f2_unpack(f2_fma(f2_add(f2_pack(__uint_as_float(c0), __uint_as_float(c1)), less), ss, mm), y[e], y[e + 1]);
          }
          const long long to = b * a.seq + w[u].i * a.pos + w[u].h * a.head + lane * 16;
          void* out = w[u].part ? a.out[1] : a.out[0];
          if (a.out_f32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + to);
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
          } else {
            uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + to);
            if (far_apart(sm[u] & 0xffffu, sm[u] >> 16)) {
              o[0] = far_values(words[u].x, s, m);
              o[1] = far_values(words[u].y, s, m);
              continue;
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
              o[q] = make_uint4(tc::pack_bf16x2(y[8 * q], y[8 * q + 1]), tc::pack_bf16x2(y[8 * q + 2], y[8 * q + 3]),
                                tc::pack_bf16x2(y[8 * q + 4], y[8 * q + 5]), tc::pack_bf16x2(y[8 * q + 6], y[8 * q + 7]));
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTok = 16;           // tokens of a tile
constexpr int kStages = 4;         // tiles of a warp on their way
constexpr int kMaxSeqs = 1024;     // sequences of a launch
constexpr int kMaxCtas = 640;
constexpr int kMaxWarps = kMaxCtas * kWarps;
constexpr int kList = 16;          // segments that a warp looks up at a time
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kNone = -3e38f;    // a reference before the first score

struct Args {
  Cache c;
  const uint16_t* q;
  long long q_seq, q_pos, q_head;
  const int32_t* lens;
  const int32_t* kpr;
  int window, sinks;
  float scale;  // times log2(e)
  uint16_t* out;
  long long o_seq, o_pos, o_head;
  float* lse;
  int B, K, Hq, Hkv, G;
  uint32_t* flags;
  uint32_t* counters;  // [2][kMaxWarps]: finished parts of runs, and joined runs, of cut groups; 0 between calls
  float* parts;        // [warp][2][rows * (D + 2)]
  long long clocks;    // of a wait for a copy; 0: none is waited for
};

// ROWS query rows a block: 4 (a column of the product is then a row and half of the tile's tokens
// for everything between the two products), 8 or 16.
template <int D, int ROWS>
struct Shape {
  static constexpr int kRows = ROWS;
  static constexpr int NT = ROWS == 16 ? 2 : 1;
  static constexpr int kUnroll = NT == 1 ? 2 : 1;  // tiles a turn
  static constexpr int kRowBytes = D / 2;
  static constexpr int kTileBytes = 2 * kTok * kRowBytes + 2 * kTok * 4;  // K, V, (s, m) of both
  static constexpr int kRing = kWarps * kStages * kTileBytes;
  static constexpr int kPart = kRows * (D + 2);  // floats of a part in memory
  // Two tiles a turn want 160 registers; so do two blocks of columns of 64 (32 sequences of up to 8192 tokens, 8 heads
  // of 64, 40 rows a group: 83 us with two CTAs an SM, 71 with three), of 128 they want 230 (163 us against 176).
  static constexpr int kMinCtas = NT == 1 || D == 64 ? 3 : 2;
  // shared memory beside the ring: lists, barriers, and the fragments of Q of two blocks of columns (bytes, about)
  static constexpr int kStatic = 5000 + kWarps * (kRows * D * 2 + (NT == 1 ? 0 : NT * D * 16));
};

// One sequence: what its queries see, in tiles.
struct Seq {
  int len, k;
  int sink_tiles, skip;  // tiles below sink_tiles, then those from sink_tiles + skip on
  int tiles, blocks;     // key tiles (one at least), blocks of query rows
  uint32_t bad;
};
__device__ __forceinline__ Seq seq_of(const Args& a, int b, int rows) {
  Seq s;
  s.len = a.lens[b];
  s.k = a.kpr ? a.kpr[b] : a.K;
  s.bad = 0;
  if (s.k < 0 || s.k > a.K) {
    s.bad = SV_FLAG_BAD_K;
    s.k = a.K;
  } else if (s.len < 0 || (long long)s.len + s.k > (long long)a.c.max_pages * a.c.page_size) {
    s.bad = SV_FLAG_BAD_N;
  }
  s.sink_tiles = s.skip = 0;
  s.tiles = 1;
  s.blocks = (a.G * (s.k + 1) + rows - 1) / rows;
  if (!s.bad) {
    const int end = s.len + s.k, all = (int)(((long long)end + kTok - 1) / kTok);
    if (a.window > 0) {
      const int first = max(0, s.len - a.window) / kTok;  // of the first query's window
      s.sink_tiles = min(first, (int)(((long long)min(a.sinks, end) + kTok - 1) / kTok));
      s.skip = first - s.sink_tiles;
    }
    s.tiles = max(1, all - s.skip);
  }
  return s;
}

// A warp's run of tiles of one group (sequence b, key head h, block of query rows).
struct Segment {
  Seq s;
  int b, h, block, t0, t1;
  unsigned long long group;  // where the group begins, in units of a tile's cost

  __device__ __forceinline__ int count() const { return s.bad || s.len + s.k == 0 ? 0 : t1 - t0; }
};

// Where the sequences' groups begin, by cost and by number, and what one costs.
struct Books {
  unsigned long long* cost;  // [B + 1]
  uint32_t* groups;          // [B + 1]
  uint32_t* each;            // [B]
  static constexpr int kBytes = 16;  // of a sequence
};

// The number of the group that unit `at` lies in.
__device__ __forceinline__ uint32_t group_at(const Books& k, int B, unsigned long long at) {
  int lo = 0, hi = B - 1;  // the last b with cost[b] <= at
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (k.cost[mid] <= at) lo = mid; else hi = mid - 1;
  }
  return k.groups[lo] + (uint32_t)quotient(at - k.cost[lo], k.each[lo]);
}

// The runs of the warp's share [begin, end) in the groups first .. first + kList - 1, a lane per group;
// those without a tile are left out.  Returns their number; *more: whether groups follow.
__device__ __forceinline__ int list_segments(const Args& a, const Books& k, int rows, uint32_t first,
                                             unsigned long long begin, unsigned long long end, int lane, Segment* list,
                                             bool* more) {
  Segment g;
  g.t0 = g.t1 = 0;
  bool goes_on = false;
  if (lane < kList && first + lane < k.groups[a.B]) {
    const uint32_t number = first + lane;
    int lo = 0, hi = a.B - 1;  // the last b with groups[b] <= number
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (k.groups[mid] <= number) lo = mid; else hi = mid - 1;
    }
    g.b = lo;
    g.s = seq_of(a, lo, rows);
    const uint32_t group = number - k.groups[lo], cost = k.each[lo];
    g.group = k.cost[lo] + (unsigned long long)group * cost;
    g.h = (int)(group / (uint32_t)g.s.blocks);
    g.block = (int)(group - (uint32_t)g.h * g.s.blocks);
    if (g.group < end) {
      g.t0 = begin > g.group ? max(0, (int)(begin - g.group) - kGroupCost) : 0;
      g.t1 = max(0, (int)min((unsigned long long)cost, end - g.group) - kGroupCost);
    }
    goes_on = g.group + cost < end;
  }
  const unsigned some = __ballot_sync(kFull, g.t0 < g.t1);
  *more = __ballot_sync(kFull, goes_on) >> (kList - 1) & 1;
  __syncwarp();  // (the list before is read no more)
  if (g.t0 < g.t1) list[__popc(some & ((1u << lane) - 1u))] = g;
  __syncwarp();
  return __popc(some);
}

// zeros in place of what is not there
__device__ __forceinline__ void cp16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(p) : "memory");
  return v;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float log2_of(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;

__device__ __forceinline__ void bulk(uint32_t to, const void* from, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
               "l"(from), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}
// A wait of at most about a second; none at all if `clocks` is 0.
__device__ __forceinline__ bool arrived(uint64_t* bar, uint32_t parity, long long clocks) {
  return clocks > 0 && tc::wait_bounded(bar, parity, clocks);
}

// The loads of a warp's tiles into its ring, in the order of the list's segments: they run ahead of the
// products, over the ends of segments too.  A page of whole tiles has a tile's four pieces (codes and
// (s, m) of K and V) as runs of bytes, one run if the page is a tile: bulk copies.  Lane l looks up and
// asks for the l-th tile of a batch of 32 (or what the segment has left), so that a tile costs the warp a
// dozen instructions (a copy per 16 bytes and lane: some fifty); the next batch's page ids are read
// while one is asked for.
template <int D, bool ALIGNED, int U>  // U tiles are taken at a time, so at most kStages - U more are on their way
struct Loader;

template <int D, int U>
struct Loader<D, true, U> {
  static constexpr int RB = D / 2;
  static constexpr uint32_t TB = 2 * kTok * RB + 2 * kTok * 4;
  const Segment* list;
  uint64_t* bars;
  uint32_t ring;         // of the warp
  int segments;
  uint32_t bad;          // a bit per segment: a page that is not there
  int i, batch;          // tiles of the batch: asked for, all
  const uint8_t* src;    // this lane's tile's K codes; NULL: a page that is not there
  int words;             // from there to K's (s, m)
  int next, base, page;  // the next batch: its segment, its first tile's number there, this lane's page
  uint32_t asked, taken; // over all segments
  bool dead;             // a wait ran out

  __device__ __forceinline__ void init(const Segment* list_, uint64_t* bars_, uint32_t ring_, int lane) {
    list = list_, bars = bars_, ring = ring_;
    asked = taken = 0;
    dead = false;
    if (lane < kStages) mbar_init(bars + lane, 1);
    fence_mbar_init();
  }
  __device__ __forceinline__ int token(const Segment& g, int lane) const {
    const int tile = g.t0 + base + lane;
    return (tile + (tile < g.s.sink_tiles ? 0 : g.s.skip)) * kTok;
  }
  __device__ __forceinline__ void look_up(const Args& a, int lane) {
    while (next < segments && base >= list[next].count()) ++next, base = 0;
    page = -1;
    if (next < segments && base + lane < list[next].count()) {
      const Segment& g = list[next];
      page = a.c.table[(long long)g.b * a.c.max_pages + divide(token(g, lane), a.c.by_page)];
    }
  }
  __device__ __forceinline__ void begin(const Args& a, int segments_, int lane) {
    segments = segments_;
    bad = 0;
    i = batch = next = base = 0;
    look_up(a, lane);
  }
  __device__ __forceinline__ void issue(const Args& a, int lane) {
    if (dead) return;
    if (i == batch) {
      if (next >= segments) return;
      const Segment& g = list[next];
      batch = min(32, g.count() - base);
      i = 0;
      src = nullptr;
      if (lane < batch) {
        const int tok = token(g, lane), slot = tok - divide(tok, a.c.by_page) * a.c.page_size;
        if ((unsigned)page < (unsigned)a.c.num_pages)
          src = a.c.pool + page * a.c.page_bytes + (long long)g.h * a.c.head_bytes + slot * RB;
        else
          bad |= 1u << next;
        words = a.c.page_size * D + slot * (4 - RB);
      }
      base += 32;
      look_up(a, lane);
    }
    if (lane == i) {
      const uint32_t slot = asked & (kStages - 1), to = ring + slot * TB;
      uint64_t* bar = bars + slot;
      if (src) {
        mbar_arrive_expect_tx(bar, TB);
        if (a.c.page_size == kTok) {
          bulk(to, src, TB, bar);
        } else {
          bulk(to, src, kTok * RB, bar);
          bulk(to + kTok * RB, src + a.c.page_size * RB, kTok * RB, bar);
          bulk(to + 2 * kTok * RB, src + words, kTok * 4, bar);
          bulk(to + 2 * kTok * RB + kTok * 4, src + words + a.c.page_size * 4, kTok * 4, bar);
        }
      } else {
        mbar_arrive(bar);
      }
    }
    ++i, ++asked;
  }
  // the next tile, once it is there (a lane whose wait runs out waits no more; the result is given up)
  __device__ __forceinline__ uint32_t take(const Args& a) {
    const uint32_t slot = taken & (kStages - 1);
    if (!dead) dead = !arrived(bars + slot, taken / kStages & 1, a.clocks);
    ++taken;
    return ring + slot * TB;
  }
  // copies of a ring that was given up come to their end before the CTA does
  __device__ __forceinline__ void leave() {
    for (uint32_t p = asked > kStages ? asked - kStages : 0; p != asked; ++p)
      tc::wait_bounded(bars + (p & (kStages - 1)), p / kStages & 1);
  }
};

// Pages of any size: a copy per 16 bytes (and per (s, m)), each from its token's own page.  One group of
// copies a call, an empty one behind the last tile.
template <int D, int U>
struct Loader<D, false, U> {
  static constexpr int RB = D / 2, CHUNKS = RB / 16, COPIES = kTok * CHUNKS / 32;
  static constexpr uint32_t TB = 2 * kTok * RB + 2 * kTok * 4;
  const Segment* list;
  uint32_t ring;
  int segments;
  uint32_t bad;
  int next, base, page;  // the next tile: its segment, its number there, the page of this lane's token
  uint32_t asked, taken;
  bool dead;

  __device__ __forceinline__ void init(const Segment* list_, uint64_t*, uint32_t ring_, int) {
    list = list_, ring = ring_;
    asked = taken = 0;
    dead = false;
  }
  // this lane's token of the next tile; -1 if no query sees it
  __device__ __forceinline__ int token(const Args& a, const Segment& g, int lane) const {
    const int tile = g.t0 + base;
    const int tok = (tile + (tile < g.s.sink_tiles ? 0 : g.s.skip)) * kTok + (lane & 15);
    return tok < g.s.len + g.s.k && (a.window <= 0 || tok >= g.s.len - a.window || tok < a.sinks) ? tok : -1;
  }
  __device__ __forceinline__ void look_up(const Args& a, int lane) {
    while (next < segments && base >= list[next].count()) ++next, base = 0;
    page = -1;
    if (next < segments) {
      const int tok = token(a, list[next], lane);
      if (tok >= 0) page = a.c.table[(long long)list[next].b * a.c.max_pages + divide(tok, a.c.by_page)];
    }
  }
  __device__ __forceinline__ void begin(const Args& a, int segments_, int lane) {
    segments = segments_;
    bad = 0;
    next = base = 0;
    look_up(a, lane);
  }
  __device__ __forceinline__ void issue(const Args& a, int lane) {
    if (next < segments) {
      const Segment& g = list[next];
      const int tok = token(a, g, lane), values = a.c.page_size * RB;
      const uint8_t* head = a.c.pool + (long long)g.h * a.c.head_bytes;
      const uint32_t buf = ring + (asked & (kStages - 1)) * TB, to = buf + lane * 16;
      long long at = -1;  // of this lane's token's codes
      int slot = 0;
      if (tok >= 0) {
        slot = tok - divide(tok, a.c.by_page) * a.c.page_size;
        if ((unsigned)page < (unsigned)a.c.num_pages) at = page * a.c.page_bytes + slot * RB;
        else bad |= 1u << next;
      }
      ++base, ++asked;
      look_up(a, lane);
#pragma unroll
      for (int j = 0; j < COPIES; ++j) {
        const long long from = __shfl_sync(kFull, at, (lane + 32 * j) / CHUNKS);
        const uint8_t* src = head + (from < 0 ? 0 : from) + lane % CHUNKS * 16;
        cp16(to + j * 512, src, from >= 0);
        cp16(to + kTok * RB + j * 512, src + values, from >= 0);
      }
      const uint8_t* word =
          head + (at < 0 ? 0 : at - slot * RB) + a.c.page_size * D + slot * 4 + (lane >= 16 ? a.c.page_size * 4 : 0);
      cp4(buf + 2 * kTok * RB + lane * 4, word, at >= 0);
    }
    cp_commit();
  }
  __device__ __forceinline__ uint32_t take(const Args&) {
    cp_wait<kStages - U>();
    __syncwarp();
    return ring + (taken++ & (kStages - 1)) * TB;
  }
  __device__ __forceinline__ void leave() { cp_wait<0>(); }
};

// The rows of a segment's Q (the key head's queries of a position, then the next position's), on their way
// into the warp's shared memory while the segment in front is computed.
template <int D, int ROWS>
struct QueryRows {
  uint16_t* to;   // [ROWS][D]
  uint64_t* bar;
  uint32_t asked;
  bool dead;

  __device__ __forceinline__ void init(uint16_t* to_, uint64_t* bar_, int lane) {
    to = to_, bar = bar_, asked = 0, dead = false;
    if (lane == 0) mbar_init(bar, 1);
    fence_mbar_init();
  }
  __device__ __forceinline__ void issue(const Args& a, const Segment& g, int lane) {
    const int row0 = g.block * ROWS, rows = g.s.bad ? 0 : min(ROWS, a.G * (g.s.k + 1) - row0);
    __syncwarp();  // (the rows before are read)
    if (lane == 0) mbar_arrive_expect_tx(bar, rows * D * 2);
    __syncwarp();
    if (lane < rows) {
      const int i = (row0 + lane) / a.G, head = g.h * a.G + (row0 + lane) % a.G;
      bulk(smem_addr(to + lane * D), a.q + g.b * a.q_seq + i * a.q_pos + head * a.q_head, D * 2, bar);
    }
    ++asked;
  }
  __device__ __forceinline__ void wait(const Args& a) {
    if (!dead) dead = !arrived(bar, (asked - 1) & 1, a.clocks);
  }
  // row r's quarter t
  __device__ __forceinline__ void read(int r, int rows, int t, uint4 (&v)[D / 32]) const {
#pragma unroll
    for (int w = 0; w < D / 32; ++w)
      v[w] = r < rows ? *reinterpret_cast<const uint4*>(to + r * D + t * (D / 4) + w * 8) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void leave() {
    if (asked) tc::wait_bounded(bar, (asked - 1) & 1);
  }
};

template <int PART>
__device__ __forceinline__ float* part_of(const Args& a, unsigned warp, unsigned long long share, unsigned long long group) {
  return a.parts + ((long long)warp * 2 + part_place(warp, share, group)) * PART;
}

// The parts of the warps first, first + step, .. (n of them) joined, in the order of the warps, for all
// rows at once: numerators of the lane's D / 32 values, and lane r's sum and reference of row r.
template <int D, int ROWS>
struct Joined {
  float num[ROWS][D / 32], l, top;

  __device__ __forceinline__ void of(const Args& a, unsigned first, unsigned step, int n, unsigned long long share,
                                     unsigned long long group, int lane) {
    constexpr int PART = ROWS * (D + 2), W = D / 32;
    const int mine = ROWS * D + lane % ROWS;  // (rows that the block does not have are read too: any values)
    top = kNone, l = 0.f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int e = 0; e < W; ++e) num[r][e] = 0.f;
    constexpr int U = ROWS == 4 ? 4 : ROWS == 8 ? 2 : 1;  // parts on their way
#pragma unroll 1
    for (int p0 = 0; p0 < n; p0 += U) {
      float ref[U], sum[U], v[U][ROWS][W];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float* part = part_of<PART>(a, first + min(p0 + u, n - 1) * step, share, group);
        ref[u] = __ldcg(part + mine);
        sum[u] = __ldcg(part + mine + ROWS);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          if constexpr (W == 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(part + r * D + lane * W));
            v[u][r][0] = x.x, v[u][r][1] = x.y, v[u][r][2] = x.z, v[u][r][3] = x.w;
          } else {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(part + r * D + lane * W));
            v[u][r][0] = x.x, v[u][r][1] = x.y;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (p0 + u >= n) break;
        const float most = fmaxf(top, ref[u]), old = ex2(top - most), f = ex2(ref[u] - most);
        top = most;
        l = __fmaf_rn(l, old, sum[u] * f);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          const float fr = __shfl_sync(kFull, f, r), or_ = __shfl_sync(kFull, old, r);
#pragma unroll
          for (int e = 0; e < W; ++e) num[r][e] = __fmaf_rn(v[u][r][e], fr, num[r][e] * or_);
        }
      }
    }
  }
};

// One more of `all` is done (with what the warp wrote before); true if it was the last, which leaves 0 (no other
// group counts at the word).
__device__ __forceinline__ bool last_of(uint32_t* counter, uint32_t all, int lane) {
  __syncwarp();
  uint32_t before = 0;
  if (lane == 0) {
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    if (before == all - 1) *counter = 0;
  }
  before = __shfl_sync(kFull, before, 0);
  __syncwarp();  // (a shuffle orders no memory: what lane 0 acquired is there for the others behind this)
  return before == all - 1;
}

__device__ __forceinline__ float log_of_sum(float top, float l) {
  return l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
}

template <int D, int ROWS, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, Shape<D, ROWS>::kMinCtas) attention_kernel(const __grid_constant__ Args a) {
  using S = Shape<D, ROWS>;
  constexpr int NT = S::NT, RB = D / 2;
  constexpr bool HALF = ROWS == 4;
  constexpr int TP = HALF ? 1 : 2;      // tokens a lane holds scores of
  constexpr int WK = D / 32;            // code words of a key per lane
  constexpr int U = S::kUnroll;
  constexpr int TILES = D / 16;         // 16-row tiles of O^T
  constexpr uint32_t TB = S::kTileBytes;
  extern __shared__ __align__(16) uint8_t smem[];
  Books books;
  books.cost = reinterpret_cast<unsigned long long*>(smem + S::kRing);
  books.groups = reinterpret_cast<uint32_t*>(books.cost + a.B + 1);
  books.each = books.groups + a.B + 1;
  __shared__ unsigned long long warp_cost[kWarps];
  __shared__ uint32_t warp_groups[kWarps];
  __shared__ Segment lists[kWarps][kList];
  __shared__ uint64_t bars[kWarps][kStages], q_bars[kWarps];
  __shared__ __align__(16) uint16_t q_rows[kWarps][ROWS * D];
  __shared__ uint2 q_frags[NT == 1 ? 1 : kWarps][NT == 1 ? 1 : NT * 2 * WK * 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  // row g of a product stands for token `tau` of its 8: pairs of rows (2t, 2t + 1), which a lane reads
  // V's codes of, are tokens t and t + 4, so that the four t's rows lie beside each other
  const int tau = (g >> 1) + (g & 1) * 4;
  // the columns of the product whose scores the lane holds: col0, col0 + 1, for tokens tok_of (+ 8)
  const int col0 = HALF ? 2 * (t & 1) : 2 * t, tok_of = HALF ? tau + (t >> 1) * 8 : tau;
  Segment* list = lists[warp];
  uint2* q_frag = q_frags[NT == 1 ? 0 : warp];
  const uint32_t q_at = smem_addr(q_frag) + lane * 8;
  Loader<D, ALIGNED, U> ld;
  ld.init(list, bars[warp], smem_addr(smem) + warp * kStages * TB, lane);
  QueryRows<D, ROWS> qr;
  qr.init(q_rows[warp], q_bars + warp, lane);
  pdl_wait();

  // the groups in a row, each as long as its tiles and kGroupCost
  {
    const int each = (a.B + kThreads - 1) / kThreads;
    unsigned long long cost = 0;
    uint32_t groups = 0;
    for (int j = 0; j < each; ++j) {
      const int b = tid * each + j;
      if (b < a.B) {
        const Seq s = seq_of(a, b, S::kRows);
        groups += (uint32_t)s.blocks * a.Hkv;
        cost += (unsigned long long)(s.tiles + kGroupCost) * s.blocks * a.Hkv;
        books.cost[b + 1] = cost;  // (within this thread's run)
        books.groups[b + 1] = groups;
        books.each[b] = (uint32_t)(s.tiles + kGroupCost);
      }
    }
    unsigned long long up = cost;
    uint32_t up_groups = groups;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const unsigned long long v = __shfl_up_sync(kFull, up, m);
      const uint32_t w = __shfl_up_sync(kFull, up_groups, m);
      if (lane >= m) up += v, up_groups += w;
    }
    if (lane == 31) warp_cost[warp] = up, warp_groups[warp] = up_groups;
    __syncthreads();
    up -= cost, up_groups -= groups;
    for (int w = 0; w < warp; ++w) up += warp_cost[w], up_groups += warp_groups[w];
    for (int j = 0; j < each; ++j) {
      const int b = tid * each + j;
      if (b < a.B) books.cost[b + 1] += up, books.groups[b + 1] += up_groups;
    }
    if (tid == 0) books.cost[0] = books.groups[0] = 0;
    __syncthreads();
  }
  // the share of this warp; from here on the warps go their own ways
  const unsigned worker = blockIdx.x * kWarps + warp;
  const unsigned long long total = books.cost[a.B];
  const unsigned long long share = share_of(total, gridDim.x * kWarps);
  const unsigned long long begin = worker * share, end = min(begin + share, total);
  if (begin >= end) return;

  bool more = true;
#pragma unroll 1
  for (uint32_t first = group_at(books, a.B, begin); more; first += kList) {
  const int segments = list_segments(a, books, S::kRows, first, begin, end, lane, list, &more);
  ld.begin(a, segments, lane);  // (page ids are on their way while Q is asked for)
  if (segments > 0) qr.issue(a, list[0], lane);
#pragma unroll 1
  for (int st = 0; st < kStages - U; ++st) ld.issue(a, lane);
#pragma unroll 1
  for (int at = 0; at < segments; ++at) {
    const Segment& sg = list[at];
    const Seq s = sg.s;
    const int row0 = sg.block * S::kRows, rows = min(S::kRows, a.G * (s.k + 1) - row0);

    // Q's rows in fp16 next to 2^15, in the order of the codes' halves; those of two blocks of columns stay
    // in shared memory (32 registers less)
    qr.wait(a);
    uint32_t qf[2 * WK][2];
    float fr[NT][2], sq[NT][2];  // of the lane's columns: score = s (acc fr) + m sq
    int limit[NT][2];      // the first token that the column's query does not see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint4 qv[WK];
      qr.read(nt * 8 + g, rows, t, qv);
      uint32_t top = 0;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        const uint32_t u[4] = {qv[w].x, qv[w].y, qv[w].z, qv[w].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          top = max(top, max(u[e] & 0x7fffu, (u[e] >> 16) & 0x7fffu));
          sum += bf16_lo(u[e]) + bf16_hi(u[e]);
        }
      }
      top = max(top, __shfl_xor_sync(kFull, top, 1));
      top = max(top, __shfl_xor_sync(kFull, top, 2));
      sum += __shfl_xor_sync(kFull, sum, 1);
      sum += __shfl_xor_sync(kFull, sum, 2);
      const int ex = (int)(top >> 7);  // biased exponent of the largest value
      // 2^(14 - its exponent), at most 2^120; NaN for a row that is not finite
      const int fb = min(268 - ex, 247);
      const float f = ex == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)fb << 23);
      const float f16 = f * 0.0625f;
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        const uint4 u = qv[w];  // values 0 1 | 2 3 | 4 5 | 6 7
        qf[2 * w][0] = half2_of(bf16_lo(u.x) * f, bf16_lo(u.z) * f);
        qf[2 * w][1] = half2_of(bf16_hi(u.x) * f16, bf16_hi(u.z) * f16);
        qf[2 * w + 1][0] = half2_of(bf16_lo(u.y) * f, bf16_lo(u.w) * f);
        qf[2 * w + 1][1] = half2_of(bf16_hi(u.y) * f16, bf16_hi(u.w) * f16);
      }
      const float mine_fr = a.scale * __uint_as_float((uint32_t)(254 - fb) << 23) * 16777216.f, mine_sq = a.scale * sum;
      if constexpr (NT > 1) {
#pragma unroll
        for (int w = 0; w < 2 * WK; ++w)  // (read by this lane alone)
          q_frag[(nt * 2 * WK + w) * 32 + lane] = make_uint2(qf[w][0], qf[w][1]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        fr[nt][j] = __shfl_sync(kFull, mine_fr, (col0 + j) * 4);
        sq[nt][j] = __shfl_sync(kFull, mine_sq, (col0 + j) * 4);
        const int col = nt * 8 + col0 + j;
        limit[nt][j] = col < rows ? s.len + (row0 + col) / a.G : 0;
      }
    }
    if (at + 1 < segments) qr.issue(a, list[at + 1], lane);
    // tiles t0 + [sure, sure + plain) are seen whole by every row of the block: those in front of the last one's
    // tokens (and behind the beginning of the last row's window)
    int sure = 0, plain = (s.len + row0 / a.G) / kTok;
    if (a.window > 0) {
      const int widest = (max(0, s.len + (row0 + rows - 1) / a.G - a.window) + kTok - 1) / kTok;
      sure = max(widest - s.skip, s.sink_tiles) - sg.t0;
      plain -= s.skip;
    }
    plain = max(0, plain - sg.t0 - sure);

    float o[NT][TILES][4] = {};
    float sum[NT][2] = {}, low[NT][2] = {};
    float ref[NT][2], vref[NT][2];  // references of p, and of 2^-7 p s', negated
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) ref[nt][0] = ref[nt][1] = vref[nt][0] = vref[nt][1] = -kNone;

    {
      // U tiles a turn: their chains of products, exponentials and products do not wait for one another
      const int n = sg.count();
#pragma unroll 1
      for (int j = 0; j < n; j += U) {
        uint32_t buf[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u == 0 || j + u < n) ld.issue(a, lane);
#pragma unroll
        for (int u = 0; u < U; ++u)  // (no tile: none of its tokens counts)
          buf[u] = u == 0 || j + u < n ? ld.take(a) : buf[0];

        float z[U][NT][TP][2], zv[U][NT][TP][2], vm[U][TP];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          // S^T: tokens tau and tau + 8 by columns 2t and 2t + 1
          float acc[NT][4] = {}, acc2[NT][4] = {};  // (two chains of products)
          uint32_t x[WK], y[WK];
          if constexpr (D == 128) {
            const uint4 p = lds128(buf[u] + tau * RB + t * 16), r = lds128(buf[u] + (tau + 8) * RB + t * 16);
            x[0] = p.x, x[1] = p.y, x[2] = p.z, x[3] = p.w;
            y[0] = r.x, y[1] = r.y, y[2] = r.z, y[3] = r.w;
          } else {
            const uint2 p = lds64(buf[u] + tau * RB + t * 8), r = lds64(buf[u] + (tau + 8) * RB + t * 8);
            x[0] = p.x, x[1] = p.y;
            y[0] = r.x, y[1] = r.y;
          }
#pragma unroll
          for (int w = 0; w < WK; ++w) {
            const uint32_t x8 = x[w] >> 8, y8 = y[w] >> 8;
            uint2 b0[NT], b1[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (NT == 1) {
                b0[nt] = make_uint2(qf[2 * w][0], qf[2 * w][1]);
                b1[nt] = make_uint2(qf[2 * w + 1][0], qf[2 * w + 1][1]);
              } else {
                b0[nt] = lds64(q_at + (nt * 2 * WK + 2 * w) * 256);
                b1[nt] = lds64(q_at + (nt * 2 * WK + 2 * w + 1) * 256);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(acc[nt], x[w] & kLow, y[w] & kLow, x[w] & kHigh, y[w] & kHigh, b0[nt].x, b0[nt].y);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(acc2[nt], x8 & kLow, y8 & kLow, x8 & kHigh, y8 & kHigh, b1[nt].x, b1[nt].y);
          }
#pragma unroll
          for (int e = 0; e < TP; ++e) {
            const uint32_t kw = lds32(buf[u] + 2 * kTok * RB + (tok_of + 8 * e) * 4);
            const uint32_t vw = lds32(buf[u] + 2 * kTok * RB + 64 + (tok_of + 8 * e) * 4);
            const float ks = bf16_lo(kw), km = bf16_hi(kw), lg = log2_of(bf16_lo(vw));
            vm[u][e] = bf16_hi(vw);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float c[2] = {acc[nt][2 * e] + acc2[nt][2 * e], acc[nt][2 * e + 1] + acc2[nt][2 * e + 1]};
              if constexpr (HALF) {  // tokens tau + 8 to the lanes of the columns that have no row
                const float c2 = __shfl_xor_sync(kFull, acc[nt][2] + acc2[nt][2], 2);
                const float c3 = __shfl_xor_sync(kFull, acc[nt][3] + acc2[nt][3], 2);
                if (t >= 2) c[0] = c2, c[1] = c3;
              }
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                z[u][nt][e][i] = __fmaf_rn(ks, c[i] * fr[nt][i], km * sq[nt][i]);
                zv[u][nt][e][i] = z[u][nt][e][i] + lg;
              }
            }
          }
        }
        const bool edge = j < sure || j + U > sure + plain || j + U > n;
        if (edge) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int tile = sg.t0 + j + u, tok0 = (tile + (tile < s.sink_tiles ? 0 : s.skip)) * kTok + tok_of;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < TP; ++e)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int lim = limit[nt][i], tok = tok0 + 8 * e;
                  const bool seen = j + u < n && tok < lim && (a.window <= 0 || tok >= lim - a.window || tok < a.sinks);
                  z[u][nt][e][i] = seen ? z[u][nt][e][i] : -INFINITY;
                  zv[u][nt][e][i] = seen ? zv[u][nt][e][i] : -INFINITY;
                }
          }
        }
        // less the references, which follow their maxima only when these have grown by 2^8
        float m[NT][2], mv[NT][2];
        bool raise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            m[nt][i] = z[0][nt][0][i], mv[nt][i] = zv[0][nt][0][i];
#pragma unroll
            for (int k = 1; k < U * TP; ++k) {
              m[nt][i] = fmaxf(m[nt][i], z[k / TP][nt][k % TP][i]);
              mv[nt][i] = fmaxf(mv[nt][i], zv[k / TP][nt][k % TP][i]);
            }
          }
          raise = raise || fmaxf(m[nt][0] + ref[nt][0], m[nt][1] + ref[nt][1]) > 8.f ||
                  fmaxf(mv[nt][0] + vref[nt][0], mv[nt][1] + vref[nt][1]) > 15.f;
        }
        if (__any_sync(kFull, raise)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float fv[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
              for (int d = HALF ? 2 : 4; d < 32; d <<= 1) {
                m[nt][i] = fmaxf(m[nt][i], __shfl_xor_sync(kFull, m[nt][i], d));
                mv[nt][i] = fmaxf(mv[nt][i], __shfl_xor_sync(kFull, mv[nt][i], d));
              }
              const float to = fminf(-m[nt][i], ref[nt][i]), tov = fminf(7.f - mv[nt][i], vref[nt][i]);
              const float f = ex2(to - ref[nt][i]);
              sum[nt][i] *= f;
              low[nt][i] *= f;
              fv[i] = ex2(tov - vref[nt][i]);
              ref[nt][i] = to;
              vref[nt][i] = tov;
            }
#pragma unroll
            for (int n = 0; n < TILES; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nt][n][e] *= fv[e & 1];
          }
        }
        uint32_t pt[U][NT][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint32_t h[TP];
#pragma unroll
            for (int e = 0; e < TP; ++e) {
              float v[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float p = ex2(z[u][nt][e][i] + ref[nt][i]);
                sum[nt][i] += p;
                // (the minimum of a token that is not seen may be anything)
                if (!edge || z[u][nt][e][i] != -INFINITY) low[nt][i] = __fmaf_rn(p, vm[u][e], low[nt][i]);
                v[i] = ex2(zv[u][nt][e][i] + vref[nt][i]);
              }
              h[e] = half2_of(v[0], v[1]);
            }
            pt[u][nt][0] = transpose8(h[0]);
            if constexpr (HALF) pt[u][nt][1] = __shfl_xor_sync(kFull, pt[u][nt][0], 16);
            else pt[u][nt][1] = transpose8(h[TP - 1]);
          }

        // O^T: pairs of tokens (t, t + 4), (t + 8, t + 12), this lane's codes of each
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t vb = buf[u] + kTok * RB;
          if constexpr (D == 128) {
            uint2 w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = lds64(vb + (t + 4 * e) * RB + g * 8);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t sel = hf ? 0x7632u : 0x5410u;
              uint32_t a0 = __byte_perm(w[0].x, w[1].x, sel), a1 = __byte_perm(w[0].y, w[1].y, sel);
              uint32_t a2 = __byte_perm(w[2].x, w[3].x, sel), a3 = __byte_perm(w[2].y, w[3].y, sel);
#pragma unroll
              for (int sh = 0; sh < 2; ++sh) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma_f16(o[nt][hf * 4 + sh * 2], a0 & kLow, a1 & kLow, a2 & kLow, a3 & kLow, pt[u][nt][0], pt[u][nt][1]);
                  mma_f16(o[nt][hf * 4 + sh * 2 + 1], a0 & kHigh, a1 & kHigh, a2 & kHigh, a3 & kHigh, pt[u][nt][0],
                          pt[u][nt][1]);
                }
                a0 >>= 8, a1 >>= 8, a2 >>= 8, a3 >>= 8;
              }
            }
          } else {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = lds32(vb + (t + 4 * e) * RB + g * 4);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t sel = hf ? 0x7632u : 0x5410u;
              uint32_t a0 = __byte_perm(w[0], w[1], sel), a2 = __byte_perm(w[2], w[3], sel);
#pragma unroll
              for (int sh = 0; sh < 2; ++sh) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_f16(o[nt][hf * 2 + sh], a0 & kLow, a0 & kHigh, a2 & kLow, a2 & kHigh, pt[u][nt][0], pt[u][nt][1]);
                a0 >>= 8, a2 >>= 8;
              }
            }
          }
        }
        __syncwarp();
      }
    }

    // the lanes' sums joined: all lanes of a column hold them
    const bool dead = __any_sync(kFull, ld.dead || qr.dead), bad = s.bad || dead || __any_sync(kFull, ld.bad >> at & 1);
    if (lane == 0 && s.bad && sg.group == books.cost[sg.b]) atomicOr(a.flags, s.bad);
    if (lane == 0 && bad && !s.bad && !dead) atomicOr(a.flags, SV_FLAG_BAD_PAGE);
    const bool whole = sg.t0 == 0 && sg.t1 == s.tiles;
    float* part = part_of<S::kPart>(a, worker, share, sg.group);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float l[2] = {sum[nt][0], sum[nt][1]}, add[2] = {low[nt][0], low[nt][1]};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int d = HALF ? 2 : 4; d < 32; d <<= 1) {
          l[j] += __shfl_xor_sync(kFull, l[j], d);
          add[j] += __shfl_xor_sync(kFull, add[j], d);
        }
        if (bad) l[j] = __uint_as_float(0x7fc00000u);
        const int r = nt * 8 + 2 * t + j;
        if (r >= rows || (HALF && t >= 2)) continue;
        // the codes' subnormals undone, and the 2^7 of the weights (here, so that a v scale next to 2^-126 is a
        // factor above it); D = 128: odd values stand 4 bits up; D = 64: the second row of a tile does
        float even = ex2(ref[nt][j] - vref[nt][j] + 7.f), inv = 1.f;
        if (whole) inv = l[j] == 0.f ? 0.f : __frcp_rn(l[j]);
        float x[TILES], y[TILES];
#pragma unroll
        for (int n = 0; n < TILES; ++n) {
          const float u0 = D == 128 && (n & 1) ? 0x1p13f : 0x1p17f, u1 = D == 128 ? u0 : 0x1p13f;
          x[n] = __fmaf_rn(o[nt][n][j] * u0, even, add[j]) * inv;
          y[n] = __fmaf_rn(o[nt][n][2 + j] * u1, even, add[j]) * inv;
        }
        // this lane's run of the row: 16g .. 16g + 15 (x, then y), or 8g .. 8g + 7 (in turn)
        if (whole) {
          const int i = (row0 + r) / a.G, head = sg.h * a.G + (row0 + r) % a.G;
          uint4* to = reinterpret_cast<uint4*>(a.out + sg.b * a.o_seq + i * a.o_pos + head * a.o_head + g * (D / 8));
          if constexpr (D == 128) {
            to[0] = make_uint4(tc::pack_bf16x2(x[0], x[1]), tc::pack_bf16x2(x[2], x[3]), tc::pack_bf16x2(x[4], x[5]),
                               tc::pack_bf16x2(x[6], x[7]));
            to[1] = make_uint4(tc::pack_bf16x2(y[0], y[1]), tc::pack_bf16x2(y[2], y[3]), tc::pack_bf16x2(y[4], y[5]),
                               tc::pack_bf16x2(y[6], y[7]));
          } else {
            to[0] = make_uint4(tc::pack_bf16x2(x[0], y[0]), tc::pack_bf16x2(x[1], y[1]), tc::pack_bf16x2(x[2], y[2]),
                               tc::pack_bf16x2(x[3], y[3]));
          }
          if (g == 0 && a.lse)
            a.lse[((long long)sg.b * (a.K + 1) + i) * a.Hq + head] = log_of_sum(-ref[nt][j], l[j]);
        } else {
          float2* to = reinterpret_cast<float2*>(part + r * D + g * (D / 8));
#pragma unroll
          for (int n = 0; n < TILES / 2; ++n) {
            if constexpr (D == 128) {
              to[n] = make_float2(x[2 * n], x[2 * n + 1]);
              to[n + 4] = make_float2(y[2 * n], y[2 * n + 1]);
            } else {
              to[2 * n] = make_float2(x[2 * n], y[2 * n]);
              to[2 * n + 1] = make_float2(x[2 * n + 1], y[2 * n + 1]);
            }
          }
          if (g == 0) {
            part[S::kRows * D + r] = -ref[nt][j];
            part[S::kRows * (D + 1) + r] = l[j];
          }
        }
      }
    }
    if (!whole) {
      // the last warp of a run joins its parts into the first's, the last of these writes the result
      const Run run = run_of(sg.group, s.tiles, share, worker);
      __syncwarp();  // (a run of one reads what its own lanes wrote)
      if (run.n == 1 || last_of(a.counters + run.first, run.n, lane)) {
        Joined<D, ROWS> all;
        all.of(a, run.first, 1, run.n, share, sg.group, lane);
        bool result = run.runs == 1;
        if (!result) {
          __syncwarp();  // (the part is read before it is written again)
          float* to = part_of<S::kPart>(a, run.first, share, sg.group);
#pragma unroll
          for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int e = 0; e < D / 32; ++e) to[r * D + lane * (D / 32) + e] = all.num[r][e];
          if (lane < ROWS) {
            to[ROWS * D + lane] = all.top;
            to[ROWS * (D + 1) + lane] = all.l;
          }
          result = last_of(a.counters + kMaxWarps + run.w0, run.runs, lane);
          if (result) all.of(a, run.w0, kJoin, (int)run.runs, share, sg.group, lane);
        }
        if (result) {
          // lane r: where row r goes, and what it is multiplied by
          const int i = (row0 + lane) / a.G, head = sg.h * a.G + (row0 + lane) % a.G;
          const long long to_mine = sg.b * a.o_seq + i * a.o_pos + head * a.o_head;
          const float inv_mine = all.l == 0.f ? 0.f : __frcp_rn(all.l);
          if (lane < rows && a.lse) a.lse[((long long)sg.b * (a.K + 1) + i) * a.Hq + head] = log_of_sum(all.top, all.l);
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            const float inv = __shfl_sync(kFull, inv_mine, r);
            uint32_t* to = reinterpret_cast<uint32_t*>(a.out + __shfl_sync(kFull, to_mine, r) + lane * (D / 32));
            if (r >= rows) continue;
#pragma unroll
            for (int e = 0; e < D / 64; ++e) to[e] = tc::pack_bf16x2(all.num[r][2 * e] * inv, all.num[r][2 * e + 1] * inv);
          }
        }
      }
    }
  }
  }
  if (__any_sync(kFull, ld.dead || qr.dead)) {
    if (lane == 0) atomicOr(a.flags, SV_FLAG_TIMEOUT);
    ld.leave();
    qr.leave();
  }
}

cudaLaunchConfig_t config(int blocks, int threads, size_t smem, void* stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

int failed(const char* what, cudaError_t e, std::string* err) {
  *err = std::string(what) + ": " + cudaGetErrorString(e);
  return SV_ERR_CUDA;
}

template <int D, int ROWS, bool ALIGNED>
int attention_t(Args a, std::string* err, void* stream) {
  using S = Shape<D, ROWS>;
  static std::atomic<int> ready[kMaxDevices];
  const int dev = current_device();
  if (dev < 0) {
    *err = "kv4_attention: no current device, or its ordinal is above 63";
    return SV_ERR_CUDA;
  }
  const size_t most = S::kRing + (kMaxSeqs + 1) * Books::kBytes;
  auto* kernel = attention_kernel<D, ROWS, ALIGNED>;
  cudaError_t e;
  if (!ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return failed("kv4_attention attribute", e, err);
    ready[dev].store(1, std::memory_order_release);
  }
  const Args all = a;
  for (int b0 = 0; b0 < all.B; b0 += kMaxSeqs) {
    a.B = all.B - b0 < kMaxSeqs ? all.B - b0 : kMaxSeqs;
    a.q = all.q + b0 * all.q_seq;
    a.c.table = all.c.table + (long long)b0 * all.c.max_pages;
    a.lens = all.lens + b0;
    a.kpr = all.kpr ? all.kpr + b0 : nullptr;
    a.out = all.out + b0 * all.o_seq;
    a.lse = all.lse ? all.lse + (long long)b0 * (all.K + 1) * all.Hq : nullptr;
    const size_t smem = S::kRing + (a.B + 1) * Books::kBytes;
    int ctas = 227 * 1024 / (int)(smem + 1024 + S::kStatic);
    ctas = ctas < S::kMinCtas ? ctas : S::kMinCtas;
    int grid = tc::num_sms() * ctas;
    if (grid > kMaxCtas) grid = kMaxCtas;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(grid, kThreads, smem, stream, &attr);
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return failed("kv4_attention launch", e, err);
  }
  return SV_OK;
}

// 9 to 16 rows fit one block of 16, whose tiles are taken apart once, or two of 8, on half as many more warps with two
// tiles a turn.  Rounds whose positions vary leave many of the second blocks empty: 64 sequences, 8 heads, 4 rows a
// position and 1 to 4 positions behind a window of 256 / 1024 / 2048 tokens take 30.8 / 45.6 / 67.5 us with blocks of
// 16 and 24.7 / 41.4 / 62.3 with 8.  With every row there it is 30.8 / 47.2 / 67.8 against 31.7 / 51.5 / 78.8, and 16
// short sequences (6 tiles a warp) take 30.8 against 26.2.
bool in_eights(const Args& a) {
  long long tokens = (long long)a.c.max_pages * a.c.page_size;
  if (a.window > 0) tokens = std::min(tokens, (long long)a.window + a.sinks + a.K + 2 * kTok);
  const long long warps = tc::num_sms() * 2LL * kWarps, tiles = tokens / kTok * a.B * a.Hkv;  // (at most)
  return tiles < warps * (a.kpr && a.K > 0 ? 40 : 7);
}

// The fewest columns that hold a call's rows; a page that begins and ends with a tile needs one look-up a tile.
template <int D>
int attention_d(const Args& a, std::string* err, void* stream) {
  const int rows = a.G * (a.K + 1);
  const bool aligned = a.c.page_size % kTok == 0;
  if (rows <= 4) return aligned ? attention_t<D, 4, true>(a, err, stream) : attention_t<D, 4, false>(a, err, stream);
  if (rows <= 8 || (rows <= 16 && in_eights(a)))
    return aligned ? attention_t<D, 8, true>(a, err, stream) : attention_t<D, 8, false>(a, err, stream);
  return aligned ? attention_t<D, 16, true>(a, err, stream) : attention_t<D, 16, false>(a, err, stream);
}

}  // namespace kv4

size_t kv4_head_bytes(int D, int page_size) { return ((size_t)page_size * (D + 8) + 15) / 16 * 16; }

constexpr size_t kKv4Counters = 256;  // behind the flag word
size_t kv4_attention_workspace_bytes(int K, int Hq, int Hkv, int D) {
  const int need = Hq / Hkv * (K + 1), rows = need <= 4 ? 4 : need <= 8 ? 8 : 16;
  return kKv4Counters + kv4::kMaxWarps * 8 + (size_t)kv4::kMaxWarps * 2 * rows * (D + 2) * 4;
}

int kv4_attention_launch(const Kv4AttentionLaunch& L, std::string* err) {
  kv4::Args a;
  a.c = kv4::cache_of(L.c, L.D);
  a.q = static_cast<const uint16_t*>(L.q);
  a.q_seq = L.q_seq;
  a.q_pos = L.q_pos;
  a.q_head = L.q_head;
  a.lens = L.lens;
  a.kpr = L.kpr;
  a.window = L.window;
  a.sinks = L.sinks;
  a.scale = L.scale * 1.4426950408889634f;
  a.out = static_cast<uint16_t*>(L.out);
  a.o_seq = L.o_seq;
  a.o_pos = L.o_pos;
  a.o_head = L.o_head;
  a.lse = L.lse;
  a.B = L.B;
  a.K = L.K;
  a.Hq = L.Hq;
  a.Hkv = L.c.Hkv;
  a.G = L.Hq / L.c.Hkv;
  uint8_t* ws = static_cast<uint8_t*>(L.workspace);
  a.clocks = L.wait_tries > 0 ? tc::kWaitClocks : 0;
  a.flags = reinterpret_cast<uint32_t*>(ws);
  a.counters = reinterpret_cast<uint32_t*>(ws + kKv4Counters);
  a.parts = reinterpret_cast<float*>(ws + kKv4Counters + kv4::kMaxWarps * 8);
  return L.D == 128 ? kv4::attention_d<128>(a, err, L.stream) : kv4::attention_d<64>(a, err, L.stream);
}

int kv4_rows_launch(const Kv4RowsLaunch& L, std::string* err) {
  kv4::RowArgs a;
  a.c = kv4::cache_of(L.c, L.D);
  a.starts = L.starts;
  a.n_per_row = L.n_per_row;
  a.in[0] = static_cast<const uint16_t*>(L.k_in);
  a.in[1] = static_cast<const uint16_t*>(L.v_in);
  a.out[0] = L.k_out;
  a.out[1] = L.v_out;
  a.seq = L.seq;
  a.pos = L.pos;
  a.head = L.head;
  a.out_f32 = L.dtype == SV_F32;
  a.B = L.B;
  a.T = L.T;
  a.Hkv = L.c.Hkv;
  a.flags = L.flags;
  // as many tokens a CTA as its threads take rows at a time
  const int at_once = kv4::kRowThreads / (L.D / 16) * kv4::kRowsAhead;
  a.tokens = at_once / (2 * L.c.Hkv) > 1 ? at_once / (2 * L.c.Hkv) : 1;
  if (a.tokens > L.T) a.tokens = L.T;
  a.by_rows = kv4::divider(2 * L.c.Hkv);
  // a row of CTAs a sequence, no more in all than keep every SM busy with several
  const long long per_seq = (L.T - 1) / a.tokens + 1LL, most = (long long)tc::num_sms() * 16;
  const int across = (int)(per_seq < most ? per_seq : most), rows = (int)(most / across);
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = kv4::config(across, kv4::kRowThreads, 0, L.stream, &attr);
  cfg.gridDim.y = (unsigned)(rows < 1 ? 1 : rows < L.B ? rows : L.B);
  auto* kernel = L.k_in ? (L.D == 128 ? kv4::append_kernel<128> : kv4::append_kernel<64>)
                        : (L.D == 128 ? kv4::read_kernel<128> : kv4::read_kernel<64>);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? SV_OK : kv4::failed(L.k_in ? "kv4_append launch" : "kv4_read launch", e, err);
}

}  // namespace sv
