// The cache of a draft held in 4 bits: its writing, its reading back, and the
// attention of a round's positions over it, with a sliding window and sinks.
//
// A token's key (and value) of one head is D codes c of 4 bits with a bf16 scale s
// and a bf16 minimum m, value m + s c.  A page holds, head by head, the codes of
// its tokens' keys, then of their values (D / 2 bytes each, the even value in a
// byte's low half), then four bytes (s, m) for each key and for each value.
//
// Attention splits all (sequence, key head, block of query rows) groups' key tiles evenly over
// the CTAs that fit the card, whatever the lengths are: a CTA's share begins and ends inside a
// group, and the CTA that is the last to finish a cut group joins its parts, in the order of
// the tokens.  Within a CTA four warps take 16-token tiles in turn, each with a softmax state
// of its own:
//   z_j = scale (s_j q.c_j + m_j sum q)      S^T = C_K Q^T, 16 tokens by 8 rows
//   o   = sum_j p_j m'_j + sum_j (p_j s'_j) c'_j       O^T = C_V^T P^T
// so that the tensor cores see the codes themselves and the scales stay in float32.  With the
// tokens on the 16-row side of mma.m16n8k16 a step of one query position (8 rows of a key
// head) wastes nothing, and codes never leave registers: 4 bits at the bottom of a half are
// the fp16 subnormal c 2^-24 (8 bits up c 2^-20), exact, so one AND makes two operands.  Q is
// fp16 with a power of two per row, which keeps bf16's 8 bits down to 2^-25 of the row's
// largest value; p_j s'_j is fp16 next to a running maximum of its own.
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <cstdint>

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
// Writing and reading.  D / 8 lanes share a row (16 bytes of it each), so a code
// word of 8 values is a lane's; a warp takes the 32 / (D / 8) heads' rows that
// stand beside each other.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;

struct RowArgs {
  Cache c;
  const int32_t* starts;
  const int32_t* n_per_row;
  const uint16_t* in[2];  // K, V
  void* out[2];
  long long seq, pos, head;  // elements
  int out_f32, B, T, Hkv;
  uint32_t* flags;
};

// The place of token i of sequence b; false (and a flag, once a sequence) if it has none.
__device__ __forceinline__ bool place(const RowArgs& a, int b, int i, bool report, int* page, int* slot) {
  const int start = a.starts[b], n = a.n_per_row ? a.n_per_row[b] : a.T;
  if (n < 0 || n > a.T || start < 0 || (long long)start + n > (long long)a.c.max_pages * a.c.page_size) {
    if (report && i == 0) atomicOr(a.flags, SV_FLAG_BAD_N);
    return false;
  }
  if (i >= n) return false;
  const int t = start + i, p = divide(t, a.c.by_page);
  *slot = t - p * a.c.page_size;
  *page = a.c.table[(long long)b * a.c.max_pages + p];
  if (*page < 0 || *page >= a.c.num_pages) {
    if (report) atomicOr(a.flags, SV_FLAG_BAD_PAGE);
    return false;
  }
  return true;
}

__device__ __forceinline__ float half_of(float x) { return 0.5f * x; }

// Codes of 8 values whose row has minimum m and scale s > 0: the nearest integers to
// (x - m) / s, ties to even.  By halves, since x - m may leave float32's range; a product
// with the reciprocal is off by an ulp or so, and the remainder (exact: the factors of c s
// have 4 and 8 bits) tells on which side of a border x lies.
__device__ __forceinline__ uint32_t encode(const float (&x)[8], float m, float s) {
  const float up = s < 0x1p-60f ? 0x1p80f : 1.f;  // (a subnormal scale's reciprocal may be infinite)
  const float hm = half_of(m), hs = half_of(s) * up, inv = __frcp_rn(hs);
  uint32_t word = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = __fmaf_rn(0.5f, x[e], -hm) * up;
    float c = rintf(fminf(t * inv, 15.f));
    const float r = __fmaf_rn(-c, hs, t), q = half_of(hs);
    const bool odd = (int)c & 1;
    c += r > q || (r == q && odd) ? 1.f : 0.f;
    c -= r < -q || (r == -q && odd) ? 1.f : 0.f;
    word |= (uint32_t)(int)fminf(fmaxf(c, 0.f), 15.f) << (4 * e);
  }
  return word;
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) append_kernel(const RowArgs a) {
  constexpr int LANES = D / 8;
  pdl_wait();
  const long long rows = (long long)a.B * a.T * 2 * a.Hkv;
  const long long stride = (long long)gridDim.x * (kRowThreads / LANES);
  const int lane = threadIdx.x % LANES;
  // (the lanes of a warp leave the loop together: `rounds` is the same for all)
  const long long first = (long long)blockIdx.x * (kRowThreads / LANES);
  for (long long base = first; base < rows; base += stride) {
    const long long row = base + threadIdx.x / LANES;
    const bool in_range = row < rows;
    const int h = in_range ? (int)(row % a.Hkv) : 0;
    const long long rest = in_range ? row / a.Hkv : 0;
    const int part = (int)(rest & 1);
    const int i = (int)((rest >> 1) % a.T), b = (int)((rest >> 1) / a.T);
    int page = 0, slot = 0;
    const bool ok = in_range && place(a, b, i, lane == 0 && h == 0 && part == 0, &page, &slot);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (ok)
      v = *reinterpret_cast<const uint4*>((part ? a.in[1] : a.in[0]) + b * a.seq + i * a.pos + h * a.head + lane * 8);
    const float x[8] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y),
                        bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
    float lo = x[0], hi = x[0];
    bool fine = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo = fminf(lo, x[e]);
      hi = fmaxf(hi, x[e]);
      fine = fine && isfinite(x[e]);
    }
#pragma unroll
    for (int m = 1; m < LANES; m <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
      const int other = __shfl_xor_sync(0xffffffffu, (int)fine, m);
      fine = fine && other;
    }
    if (!ok) continue;
    // (max - min) / 15, correctly rounded twice: a float32 quotient of values with 8 bits lies on
    // a border of bf16 only if the exact one does
    const float s = 2.f * __fdiv_rn(half_of(hi) - half_of(lo), 15.f);
    uint16_t sb = __bfloat16_as_ushort(__float2bfloat16_rn(s)), mb = (uint16_t)(__float_as_uint(lo) >> 16);
    const float sr = __uint_as_float((uint32_t)sb << 16);
    uint32_t word = 0;
    if (!fine) {
      sb = mb = 0x7fc0u;  // a token that is not finite makes the scores of the queries that see it NaN
    } else if (sr > 0.f) {
      word = encode(x, lo, sr);
    }
    uint8_t* at = a.c.pool + page * a.c.page_bytes + (long long)h * a.c.head_bytes;
    const int half = a.c.page_size * (D / 2);
    reinterpret_cast<uint32_t*>(at + (long long)part * half + (long long)slot * (D / 2))[lane] = word;
    if (lane == 0)
      reinterpret_cast<uint32_t*>(at + 2LL * half + (long long)part * a.c.page_size * 4)[slot] =
          (uint32_t)sb | (uint32_t)mb << 16;
  }
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const RowArgs a) {
  constexpr int LANES = D / 8;
  pdl_wait();
  const long long rows = (long long)a.B * a.T * 2 * a.Hkv;
  const int lane = threadIdx.x % LANES;
  for (long long row = (long long)blockIdx.x * (kRowThreads / LANES) + threadIdx.x / LANES; row < rows;
       row += (long long)gridDim.x * (kRowThreads / LANES)) {
    const int h = (int)(row % a.Hkv);
    const long long rest = row / a.Hkv;
    const int part = (int)(rest & 1);
    const int i = (int)((rest >> 1) % a.T), b = (int)((rest >> 1) / a.T);
    int page, slot;
    if (!place(a, b, i, lane == 0 && h == 0 && part == 0, &page, &slot)) continue;
    const uint8_t* at = a.c.pool + page * a.c.page_bytes + (long long)h * a.c.head_bytes;
    const int half = a.c.page_size * (D / 2);
    const uint32_t w = reinterpret_cast<const uint32_t*>(at + (long long)part * half + (long long)slot * (D / 2))[lane];
    const uint32_t sm =
        reinterpret_cast<const uint32_t*>(at + 2LL * half + (long long)part * a.c.page_size * 4)[slot];
    const float s = bf16_lo(sm), m = bf16_hi(sm);
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __fmaf_rn((float)(w >> (4 * e) & 15u), s, m);
    const long long to = b * a.seq + i * a.pos + h * a.head + lane * 8;
    void* out = part ? a.out[1] : a.out[0];
    if (a.out_f32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + to);
      o[0] = make_float4(y[0], y[1], y[2], y[3]);
      o[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + to) =
          make_uint4(tc::pack_bf16x2(y[0], y[1]), tc::pack_bf16x2(y[2], y[3]), tc::pack_bf16x2(y[4], y[5]),
                     tc::pack_bf16x2(y[6], y[7]));
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
constexpr int kMaxCtas = 1024;
constexpr int kMinTiles = 8;       // of a CTA: two a warp
constexpr uint32_t kFull = 0xffffffffu;

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
  uint32_t* counters;  // [kMaxCtas]: finished parts of the group that a CTA's share ends in; 0 between calls
  float* parts;        // [CTA][2][rows * (D + 2)]
};

template <int D, int NT>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kRowBytes = D / 2;
  static constexpr int kTileBytes = 2 * kTok * kRowBytes + 2 * kTok * 4;  // K, V, (s, m) of both
  static constexpr int kRing = kWarps * kStages * kTileBytes;
  // a row's numerators in float32, a word left out after each of a lane's runs, so that the lanes of a
  // store (rows 2t, values 16g or 8g apart) meet 32 banks
  static constexpr int kRun = D == 128 ? 16 : 8;
  static constexpr int kPitch = D == 128 ? 148 : 84;
  static constexpr int kJoin = kWarps * kRows * (kPitch + 2) * 4;
  static constexpr int kPart = kRows * (D + 2);  // floats of a part in memory
  static constexpr int kMinCtas = NT == 1 ? 4 : 3;
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

__device__ __forceinline__ void cp16(uint32_t to, const void* from, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t to, const void* from, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
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
// x - ref, 2^ of it: a reference of -inf (nothing seen yet) counts as 0
__device__ __forceinline__ float weight_of(float x, float ref) { return ex2(x - (ref == -INFINITY ? 0.f : ref)); }

constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;

// Where a warp's tile is loaded from, for this lane's token of it.
template <int D>
__device__ __forceinline__ void issue_tile(const Cache& c, const Seq& s, int tile, int lane, int b, int h, uint32_t ring,
                                           bool* bad_page) {
  constexpr int RB = D / 2, CHUNKS = RB / 16;  // 16-byte pieces of a row
  const int tok = (tile + (tile < s.sink_tiles ? 0 : s.skip)) * kTok + (lane & 15);
  long long at = -1, word = -1;
  if (tok < s.len + s.k) {
    const int p = divide(tok, c.by_page), slot = tok - p * c.page_size;
    const int page = c.table[(long long)b * c.max_pages + p];
    if (page >= 0 && page < c.num_pages) {
      const long long head = page * c.page_bytes + (long long)h * c.head_bytes;
      at = head + (long long)slot * RB;
      word = head + (long long)c.page_size * D + slot * 4LL;
    } else {
      *bad_page = true;
    }
  }
  const long long values = (long long)c.page_size * RB;
#pragma unroll
  for (int j = 0; j < kTok * CHUNKS / 32; ++j) {
    const int row = (lane + 32 * j) / CHUNKS, chunk = lane % CHUNKS;
    const long long from = __shfl_sync(kFull, at, row);
    const uint32_t bytes = from < 0 ? 0 : 16;
    const uint8_t* src = c.pool + (from < 0 ? 0 : from + chunk * 16);
    const uint32_t to = ring + row * RB + ((chunk ^ (row >> 1)) & (CHUNKS - 1)) * 16;
    cp16(to, src, bytes);
    cp16(to + kTok * RB, src + (from < 0 ? 0 : values), bytes);
  }
  const bool of_values = lane >= 16;
  cp4(ring + 2 * kTok * RB + lane * 4, c.pool + (word < 0 ? 0 : word + (of_values ? c.page_size * 4LL : 0)),
      word < 0 ? 0 : 4);
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Shape<D, NT>::kMinCtas) attention_kernel(const __grid_constant__ Args a) {
  using S = Shape<D, NT>;
  constexpr int RB = D / 2;
  constexpr int WK = D / 32;            // code words of a key per lane
  constexpr int TILES = D / 16;         // 16-row tiles of O^T
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* ring_base = smem;
  float* join = reinterpret_cast<float*>(smem + S::kRing);                   // [warp][row][pitch]
  float* join_r = join + kWarps * S::kRows * S::kPitch;                      // [warp][row]
  float* join_l = join_r + kWarps * S::kRows;
  unsigned long long* prefix = reinterpret_cast<unsigned long long*>(smem + S::kRing + S::kJoin);  // [B + 1]
  __shared__ unsigned long long warp_sum[kWarps];
  __shared__ uint32_t bad_of_cta, last_of_group;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  pdl_wait();

  // the groups' tiles in a row: prefix[b] is where sequence b's begin
  {
    const int each = (a.B + kThreads - 1) / kThreads;
    unsigned long long mine = 0;
    for (int j = 0; j < each; ++j) {
      const int b = tid * each + j;
      if (b < a.B) {
        const Seq s = seq_of(a, b, S::kRows);
        mine += (unsigned long long)s.tiles * s.blocks * a.Hkv;
        prefix[b + 1] = mine;  // (within this thread's run)
      }
    }
    unsigned long long up = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const unsigned long long v = __shfl_up_sync(kFull, up, m);
      if (lane >= m) up += v;
    }
    if (lane == 31) warp_sum[warp] = up;
    __syncthreads();
    unsigned long long before = up - mine;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    for (int j = 0; j < each; ++j) {
      const int b = tid * each + j;
      if (b < a.B) prefix[b + 1] += before;
    }
    if (tid == 0) prefix[0] = 0;
    __syncthreads();
  }
  const unsigned long long total = prefix[a.B];
  unsigned long long share = (total + gridDim.x - 1) / gridDim.x;
  if (share < kMinTiles) share = kMinTiles;
  const unsigned long long begin = blockIdx.x * share;
  const unsigned long long end = min(begin + share, total);
  const uint32_t ring = smem_addr(ring_base) + warp * kStages * S::kTileBytes;

  for (unsigned long long at = begin; at < end;) {
    // the group that `at` lies in
    int b = 0;
    {
      int lo = 0, hi = a.B - 1;  // the last b with prefix[b] <= at
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= at) lo = mid; else hi = mid - 1;
      }
      b = lo;
    }
    const Seq s = seq_of(a, b, S::kRows);
    const unsigned long long off = at - prefix[b];
    const int group = (int)(off / s.tiles);
    const int t0 = (int)(off - (unsigned long long)group * s.tiles);
    const int t1 = (int)min((unsigned long long)s.tiles, t0 + (end - at));
    const int h = group / s.blocks, block = group - h * s.blocks;
    const int row0 = block * S::kRows, rows = min(S::kRows, a.G * (s.k + 1) - row0);
    bool bad_page = false;

    // the first tiles
    int ahead = t0 + warp;
    if (!s.bad) {
#pragma unroll
      for (int st = 0; st < kStages - 1; ++st) {
        if (ahead < t1) issue_tile<D>(a.c, s, ahead, lane, b, h, ring + st * S::kTileBytes, &bad_page);
        cp_commit();
        ahead += kWarps;
      }
    }

    // Q's rows in fp16 next to 2^15, in the order of the codes' halves
    uint32_t qf[NT][2 * WK][2];
    float fr[NT][2], sq[NT][2];  // of the columns 2t, 2t + 1: score = s (acc fr) + m sq
    int limit[NT][2];            // the first token that the column's query does not see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
      uint4 v[WK];
#pragma unroll
      for (int w = 0; w < WK; ++w) v[w] = make_uint4(0, 0, 0, 0);
      if (r < rows && !s.bad) {
        const int i = (row0 + r) / a.G, head = h * a.G + (row0 + r) % a.G;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + b * a.q_seq + i * a.q_pos + head * a.q_head + t * (D / 4));
#pragma unroll
        for (int w = 0; w < WK; ++w) v[w] = __ldg(src + w);
      }
      uint32_t top = 0;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        const uint32_t u[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
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
        const uint4 u = v[w];  // values 0 1 | 2 3 | 4 5 | 6 7
        qf[nt][2 * w][0] = half2_of(bf16_lo(u.x) * f, bf16_lo(u.z) * f);
        qf[nt][2 * w][1] = half2_of(bf16_hi(u.x) * f16, bf16_hi(u.z) * f16);
        qf[nt][2 * w + 1][0] = half2_of(bf16_lo(u.y) * f, bf16_lo(u.w) * f);
        qf[nt][2 * w + 1][1] = half2_of(bf16_hi(u.y) * f16, bf16_hi(u.w) * f16);
      }
      const float mine_fr = a.scale * __uint_as_float((uint32_t)(254 - fb) << 23) * 16777216.f, mine_sq = a.scale * sum;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        fr[nt][j] = __shfl_sync(kFull, mine_fr, (2 * t + j) * 4);
        sq[nt][j] = __shfl_sync(kFull, mine_sq, (2 * t + j) * 4);
        const int col = nt * 8 + 2 * t + j;
        limit[nt][j] = col < rows ? s.len + (row0 + col) / a.G : 0;
      }
    }
    // tokens below this are seen by every row of the block, if no window hides them
    const int all_see = s.len + row0 / a.G;
    const int widest = s.len + (row0 + rows - 1) / a.G - a.window;  // the last row's window begins here

    float o[NT][TILES][4] = {};
    float sum[NT][2] = {}, low[NT][2] = {};
    float ref[NT][2], vref[NT][2];  // references of p and of p s'
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) ref[nt][j] = vref[nt][j] = -INFINITY;

    if (!s.bad) {
      int stage = 0;
      for (int tile = t0 + warp; tile < t1; tile += kWarps) {
        const uint32_t buf = ring + stage * S::kTileBytes;
        if (ahead < t1)
          issue_tile<D>(a.c, s, ahead, lane, b, h, ring + ((stage + kStages - 1) & (kStages - 1)) * S::kTileBytes, &bad_page);
        cp_commit();
        ahead += kWarps;
        cp_wait<kStages - 1>();
        __syncwarp();

        const int tok0 = (tile + (tile < s.sink_tiles ? 0 : s.skip)) * kTok;
        const uint32_t kw0 = lds32(buf + 2 * kTok * RB + g * 4), kw1 = lds32(buf + 2 * kTok * RB + (g + 8) * 4);
        const uint32_t vw0 = lds32(buf + 2 * kTok * RB + (16 + g) * 4), vw1 = lds32(buf + 2 * kTok * RB + (24 + g) * 4);

        // S^T: tokens g and g + 8 by rows 2t and 2t + 1
        float acc[NT][4] = {};
        {
          uint32_t x[WK], y[WK];
          if constexpr (D == 128) {
            const uint4 p = lds128(buf + g * RB + ((t ^ (g >> 1)) & 3) * 16);
            const uint4 r = lds128(buf + (g + 8) * RB + ((t ^ ((g + 8) >> 1)) & 3) * 16);
            x[0] = p.x, x[1] = p.y, x[2] = p.z, x[3] = p.w;
            y[0] = r.x, y[1] = r.y, y[2] = r.z, y[3] = r.w;
          } else {
            const uint2 p = lds64(buf + g * RB + (((t >> 1) ^ (g >> 1)) & 1) * 16 + (t & 1) * 8);
            const uint2 r = lds64(buf + (g + 8) * RB + (((t >> 1) ^ ((g + 8) >> 1)) & 1) * 16 + (t & 1) * 8);
            x[0] = p.x, x[1] = p.y;
            y[0] = r.x, y[1] = r.y;
          }
#pragma unroll
          for (int w = 0; w < WK; ++w) {
            const uint32_t x8 = x[w] >> 8, y8 = y[w] >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(acc[nt], x[w] & kLow, y[w] & kLow, x[w] & kHigh, y[w] & kHigh, qf[nt][2 * w][0], qf[nt][2 * w][1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(acc[nt], x8 & kLow, y8 & kLow, x8 & kHigh, y8 & kHigh, qf[nt][2 * w + 1][0], qf[nt][2 * w + 1][1]);
          }
        }

        const float ks0 = bf16_lo(kw0), km0 = bf16_hi(kw0), ks1 = bf16_lo(kw1), km1 = bf16_hi(kw1);
        const float vm0 = bf16_hi(vw0), vm1 = bf16_hi(vw1);
        const float lg0 = log2_of(bf16_lo(vw0)), lg1 = log2_of(bf16_lo(vw1));
        const bool edge = tok0 + kTok > all_see || (a.window > 0 && tok0 < widest && tok0 + kTok > a.sinks);
        uint32_t pt[NT][2];
        bool raise = false;
        float z[NT][4], zv[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            z[nt][j] = __fmaf_rn(ks0, acc[nt][j] * fr[nt][j], km0 * sq[nt][j]);
            z[nt][2 + j] = __fmaf_rn(ks1, acc[nt][2 + j] * fr[nt][j], km1 * sq[nt][j]);
          }
          if (edge) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tok = tok0 + g + (e >> 1) * 8, lim = limit[nt][e & 1];
              const bool seen = tok < lim && (a.window <= 0 || tok >= lim - a.window || tok < a.sinks);
              z[nt][e] = seen ? z[nt][e] : -INFINITY;
              zv[nt][e] = seen ? z[nt][e] + (e < 2 ? lg0 : lg1) : -INFINITY;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) zv[nt][e] = z[nt][e] + (e < 2 ? lg0 : lg1);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            raise = raise || z[nt][e] > ref[nt][e & 1] + 8.f || zv[nt][e] > vref[nt][e & 1] + 8.f;
        }
        // a reference follows its maximum only when that has grown by 2^8
        if (__any_sync(kFull, raise)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float m = fmaxf(z[nt][j], z[nt][2 + j]), mv = fmaxf(zv[nt][j], zv[nt][2 + j]);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) {
                m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
                mv = fmaxf(mv, __shfl_xor_sync(kFull, mv, d));
              }
              if (m > ref[nt][j]) {
                const float f = ex2(ref[nt][j] - m);
                sum[nt][j] *= f;
                low[nt][j] *= f;
                ref[nt][j] = m;
              }
              if (mv > vref[nt][j]) {
                const float f = ex2(vref[nt][j] - mv);
                vref[nt][j] = mv;
#pragma unroll
                for (int n = 0; n < TILES; ++n) {
                  o[nt][n][j] *= f;
                  o[nt][n][2 + j] *= f;
                }
              }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pv[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = weight_of(z[nt][e], ref[nt][e & 1]);
            sum[nt][e & 1] += p;
            // (a token that is not seen may have any minimum)
            low[nt][e & 1] = p == 0.f ? low[nt][e & 1] : __fmaf_rn(p, e < 2 ? vm0 : vm1, low[nt][e & 1]);
            pv[e] = weight_of(zv[nt][e] + 7.f, vref[nt][e & 1]);
          }
          pt[nt][0] = transpose8(half2_of(pv[0], pv[1]));
          pt[nt][1] = transpose8(half2_of(pv[2], pv[3]));
        }

        // O^T: pairs of tokens (2t, 2t + 1), (2t + 8, 2t + 9), this lane's codes of each
        const uint32_t vb = buf + kTok * RB;
        if constexpr (D == 128) {
          uint2 w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = 2 * t + (e & 1) + (e >> 1) * 8;
            w[e] = lds64(vb + tok * RB + (((g >> 1) ^ (tok >> 1)) & 3) * 16 + (g & 1) * 8);
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t sel = hf ? 0x7632u : 0x5410u;
            uint32_t a0 = __byte_perm(w[0].x, w[1].x, sel), a1 = __byte_perm(w[0].y, w[1].y, sel);
            uint32_t a2 = __byte_perm(w[2].x, w[3].x, sel), a3 = __byte_perm(w[2].y, w[3].y, sel);
#pragma unroll
            for (int sh = 0; sh < 2; ++sh) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_f16(o[nt][hf * 4 + sh * 2], a0 & kLow, a1 & kLow, a2 & kLow, a3 & kLow, pt[nt][0], pt[nt][1]);
                mma_f16(o[nt][hf * 4 + sh * 2 + 1], a0 & kHigh, a1 & kHigh, a2 & kHigh, a3 & kHigh, pt[nt][0], pt[nt][1]);
              }
              a0 >>= 8, a1 >>= 8, a2 >>= 8, a3 >>= 8;
            }
          }
        } else {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = 2 * t + (e & 1) + (e >> 1) * 8;
            w[e] = lds32(vb + tok * RB + (((g >> 2) ^ (tok >> 1)) & 1) * 16 + (g & 3) * 4);
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t sel = hf ? 0x7632u : 0x5410u;
            uint32_t a0 = __byte_perm(w[0], w[1], sel), a2 = __byte_perm(w[2], w[3], sel);
#pragma unroll
            for (int sh = 0; sh < 2; ++sh) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(o[nt][hf * 2 + sh], a0 & kLow, a0 & kHigh, a2 & kLow, a2 & kHigh, pt[nt][0], pt[nt][1]);
              a0 >>= 8, a2 >>= 8;
            }
          }
        }
        __syncwarp();
        stage = (stage + 1) & (kStages - 1);
      }
      cp_wait<0>();
    }

    // join the warps' states
    if (tid == 0) bad_of_cta = 0;
    __syncthreads();  // (also: the join's words of the segment before have been read)
    if (s.bad || bad_page) bad_of_cta = 1;
    if (tid == 0 && s.bad && at == prefix[b]) atomicOr(a.flags, s.bad);
    if (bad_page && lane < 16) atomicOr(a.flags, SV_FLAG_BAD_PAGE);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          sum[nt][j] += __shfl_xor_sync(kFull, sum[nt][j], d);
          low[nt][j] += __shfl_xor_sync(kFull, low[nt][j], d);
        }
        if (g == 0) join_r[warp * S::kRows + nt * 8 + 2 * t + j] = ref[nt][j];
      }
    __syncthreads();
    const bool bad = bad_of_cta != 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = nt * 8 + 2 * t + j;
        float top = join_r[r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, join_r[w * S::kRows + r]);
        const float scale = weight_of(ref[nt][j], top);
        if (g == 0) join_l[warp * S::kRows + r] = sum[nt][j] * scale;
        const float add = low[nt][j] * scale;
        // codes' subnormals and the weights' 2^7 undone; nothing was seen if the reference is -inf
        const float even = vref[nt][j] == -INFINITY ? 0.f : ex2(vref[nt][j] - ref[nt][j]) * scale;
        float* to = join + (warp * S::kRows + r) * S::kPitch;
#pragma unroll
        for (int n = 0; n < TILES; ++n) {
          const int d0 = D == 128 ? 16 * g + n : 8 * g + 2 * n, d1 = D == 128 ? d0 + 8 : d0 + 1;
          // D = 128: odd values stand 4 bits up; D = 64: the second row of a tile does
          const float u0 = D == 128 && (n & 1) ? 0x1p13f : 0x1p17f, u1 = D == 128 ? u0 : 0x1p13f;
          to[d0 + d0 / S::kRun] = __fmaf_rn(o[nt][n][j] * u0, even, add);
          to[d1 + d1 / S::kRun] = __fmaf_rn(o[nt][n][2 + j] * u1, even, add);
        }
      }
    __syncthreads();

    const bool whole = t0 == 0 && t1 == s.tiles;
    const unsigned long long group_begin = at - t0, group_end = group_begin + s.tiles;
    float* part = a.parts + ((long long)blockIdx.x * 2 + (at == begin ? 0 : 1)) * S::kPart;
    for (int x = tid; x < rows * (D / 2); x += kThreads) {
      const int r = x / (D / 2), d = (x % (D / 2)) * 2;
      float n0 = 0.f, n1 = 0.f, l = 0.f, top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* from = join + (w * S::kRows + r) * S::kPitch + d + d / S::kRun;
        n0 += from[0];
        n1 += from[1];
        l += join_l[w * S::kRows + r];
        top = fmaxf(top, join_r[w * S::kRows + r]);
      }
      if (bad) l = __uint_as_float(0x7fc00000u);
      if (whole) {
        const int i = (row0 + r) / a.G, head = h * a.G + (row0 + r) % a.G;
        const float inv = l == 0.f ? 0.f : __frcp_rn(l);
        *reinterpret_cast<uint32_t*>(a.out + b * a.o_seq + i * a.o_pos + head * a.o_head + d) =
            tc::pack_bf16x2(n0 * inv, n1 * inv);
        if (d == 0 && a.lse)
          a.lse[((long long)b * (a.K + 1) + i) * a.Hq + head] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
      } else {
        part[r * D + d] = n0;
        part[r * D + d + 1] = n1;
        if (d == 0) {
          part[S::kRows * D + r] = top;
          part[S::kRows * (D + 1) + r] = l;
        }
      }
    }
    if (!whole) {
      // the last of the group's CTAs joins its parts
      const unsigned first = (unsigned)(group_begin / share), last = (unsigned)((group_end - 1) / share);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const uint32_t before = atomicAdd(a.counters + first, 1u);
        last_of_group = before == last - first;
        if (last_of_group) {
          a.counters[first] = 0;
          __threadfence();
        }
      }
      __syncthreads();
      if (last_of_group) {
        constexpr int PER = kThreads / S::kRows, W = D / PER;  // threads of a row, values of a thread
        const int r = tid / PER, d0 = (tid % PER) * W;
        const bool at_begin = group_begin == (unsigned long long)first * share;
        auto part_of = [&](unsigned c) {
          return a.parts + ((long long)c * 2 + (c == first && !at_begin ? 1 : 0)) * S::kPart;
        };
        if (r < rows) {
          float top = -INFINITY;
          for (unsigned c = first; c <= last; ++c) top = fmaxf(top, __ldcg(part_of(c) + S::kRows * D + r));
          float l = 0.f, n[W] = {};
          for (unsigned c = first; c <= last; ++c) {
            const float* p = part_of(c);
            const float f = weight_of(__ldcg(p + S::kRows * D + r), top);
            l = __fmaf_rn(__ldcg(p + S::kRows * (D + 1) + r), f, l);
#pragma unroll
            for (int e = 0; e < W; e += 4) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(p + r * D + d0 + e));
              n[e] = __fmaf_rn(v.x, f, n[e]);
              n[e + 1] = __fmaf_rn(v.y, f, n[e + 1]);
              n[e + 2] = __fmaf_rn(v.z, f, n[e + 2]);
              n[e + 3] = __fmaf_rn(v.w, f, n[e + 3]);
            }
          }
          const int i = (row0 + r) / a.G, head = h * a.G + (row0 + r) % a.G;
          const float inv = l == 0.f ? 0.f : __frcp_rn(l);
          uint32_t* to = reinterpret_cast<uint32_t*>(a.out + b * a.o_seq + i * a.o_pos + head * a.o_head + d0);
#pragma unroll
          for (int e = 0; e < W / 2; ++e) to[e] = tc::pack_bf16x2(n[2 * e] * inv, n[2 * e + 1] * inv);
          if (d0 == 0 && a.lse)
            a.lse[((long long)b * (a.K + 1) + i) * a.Hq + head] =
                l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
        }
      }
    }
    at += t1 - t0;
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

template <int D, int NT>
int attention_t(Args a, std::string* err, void* stream) {
  using S = Shape<D, NT>;
  static std::atomic<int> ready[kMaxDevices];
  const int dev = current_device();
  if (dev < 0) {
    *err = "kv4_attention: no current device, or its ordinal is above 63";
    return SV_ERR_CUDA;
  }
  const size_t most = S::kRing + S::kJoin + (kMaxSeqs + 1) * 8;
  auto* kernel = attention_kernel<D, NT>;
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
    const size_t smem = S::kRing + S::kJoin + (a.B + 1) * 8;
    int ctas = 227 * 1024 / (int)(smem + 1024);
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

}  // namespace kv4

size_t kv4_head_bytes(int D, int page_size) { return ((size_t)page_size * (D + 8) + 15) / 16 * 16; }

constexpr size_t kKv4Counters = 256;  // behind the flag word
size_t kv4_attention_workspace_bytes(int K, int Hq, int Hkv, int D) {
  const int rows = Hq / Hkv * (K + 1) > 8 ? 16 : 8;
  return kKv4Counters + kv4::kMaxCtas * 4 + (size_t)kv4::kMaxCtas * 2 * rows * (D + 2) * 4;
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
  a.flags = reinterpret_cast<uint32_t*>(ws);
  a.counters = reinterpret_cast<uint32_t*>(ws + kKv4Counters);
  a.parts = reinterpret_cast<float*>(ws + kKv4Counters + kv4::kMaxCtas * 4);
  const bool wide = a.G * (L.K + 1) > 8;
  if (L.D == 128) return wide ? kv4::attention_t<128, 2>(a, err, L.stream) : kv4::attention_t<128, 1>(a, err, L.stream);
  return wide ? kv4::attention_t<64, 2>(a, err, L.stream) : kv4::attention_t<64, 1>(a, err, L.stream);
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
  const int per = kv4::kRowThreads / (L.D / 8);
  long long blocks = ((long long)L.B * L.T * 2 * L.c.Hkv + per - 1) / per;
  const long long most = (long long)tc::num_sms() * 64;
  if (blocks > most) blocks = most;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = kv4::config((int)blocks, kv4::kRowThreads, 0, L.stream, &attr);
  auto* kernel = L.k_in ? (L.D == 128 ? kv4::append_kernel<128> : kv4::append_kernel<64>)
                        : (L.D == 128 ? kv4::read_kernel<128> : kv4::read_kernel<64>);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? SV_OK : kv4::failed(L.k_in ? "kv4_append launch" : "kv4_read launch", e, err);
}

}  // namespace sv
