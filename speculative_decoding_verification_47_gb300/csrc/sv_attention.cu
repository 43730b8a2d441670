// Attention of a round's query positions over a prefix that the whole batch
// shares and over each sequence's own tokens in a paged cache.
//
//   out = sum_j exp(s_j) v_j / sum_j exp(s_j),  s_j = scale q . k_j
//
// A softmax over a set of keys splits into softmaxes over parts of it: with the
// part's maximum m_p, l_p = sum exp(s - m_p) and o_p = sum exp(s - m_p) v,
//   out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p   (m in base 2, M the largest m_p).
// So the prefix is one matrix product for ALL query rows of a key head (rows
// (sequence, position, head of the group), 256 to an item), and only the own
// tokens are read per sequence.
//
// Three kernels on the caller's stream, chained by programmatic launches:
//  1. plan_kernel: lengths and draft counts live on the device, so the list of
//     items does too: compact query rows, chunks of long sequences, splits of the
//     prefix, sized so that the card is filled and the partial results stay bounded.
//  2. part_kernel: persistent, one CTA per SM.  An item is up to 256 query rows
//     (two streams of 128) over a run of keys in tiles of 128: S = Q K^T and
//     O += P V with tcgen05, S, P and O in tensor memory, K and V through a ring of
//     tiles in shared memory.  Pages of a power of two from 8 tokens on arrive as
//     boxes of the TMA engine; other pages row by row in 16-byte asynchronous copies.
//     With 128 rows or fewer the two streams take alternate key tiles instead.
//  3. merge_kernel: the parts of each row, in a fixed order, to out and lse.
//
// Measured with 32 query and 8 key heads of 128.  256 sequences with 2 to 8 drafts and
// 128 to 4096 own tokens behind a prefix of 16384: about 660 us; their own tokens alone 405 us
// (bound by HBM, 5.4 TB/s), the prefix alone 432 us (a stream's softmax and its products
// alternate).  64 sequences x 8 behind 2048 tokens, 100 to 511 own ones: 60 us, one token
// behind 256 and 100: 15 us (bound by latencies: the plan 3 us, the first item's Q and
// tiles 5, an item's end 1 to 2, the merge 4 to 8).
#include <cstdint>

#include "sv_internal.h"
#include "sv_tc.cuh"

namespace sv {
namespace att {

constexpr int kTileKeys = 128;
constexpr int kItemRows = 256;
constexpr int kMaxGrid = 160;  // CTAs that the partial results are sized for
constexpr int kSlack = 4;      // items per CTA that splitting aims at
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.69314718055994531f;

// Workspace header (32-bit words); word 0 is the flag word.
enum { H_FLAGS, H_ALL_FAIL, H_NEXT_PRE, H_NEXT_OWN, H_QUERIES, H_CHUNKS, H_CHUNK_KEYS, H_SPLITS, H_SPLIT_TILES,
       H_PRE_ITEMS, H_OWN_ITEMS, H_PRE_CTAS, H_WORDS = 64 };

struct Layout {  // byte offsets into the workspace
  size_t qrow, chunk_of, stat, nan_from, pre_ml, pre_o, extra_ml, extra_o, own_ml, own_o, total;
  long long pre_rows, extra_rows, own_slots;
};

__host__ inline Layout layout(int B, int K, int Hq, int Hkv, int D, long long prefix_len, long long max_own) {
  Layout w;
  const long long Q = (long long)B * (K + 1), G = Hq / Hkv, own_rows = (K + 1) * G;
  const long long ptiles = (prefix_len + kTileKeys - 1) / kTileKeys;
  const long long rt = (own_rows + kItemRows - 1) / kItemRows;
  // splits * items <= items + kSlack * grid, and a split has a tile at least
  const long long by_items = Q * Hq + (long long)kSlack * kMaxGrid * kItemRows, by_tiles = ptiles * Q * Hq;
  w.pre_rows = by_items < by_tiles ? by_items : by_tiles;
  const long long e_items = (long long)Hkv + kSlack * kMaxGrid, e_tiles = ptiles * Hkv;
  w.extra_rows = 128 * (e_items < e_tiles ? e_items : e_tiles);
  const long long c_items = B + (long long)kSlack * kMaxGrid / (Hkv * rt) + 1,
                  c_tiles = B * ((max_own + 2 * kTileKeys - 1) / (2 * kTileKeys));
  w.own_slots = (c_items < c_tiles ? c_items : c_tiles) * Hkv * 2;
  size_t at = H_WORDS * 4;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 255) / 256 * 256;
    return here;
  };
  w.qrow = take((size_t)Q * 16);
  w.chunk_of = take((size_t)(w.own_slots / (2 * Hkv)) * 16);
  w.stat = take((size_t)B * 4);
  w.nan_from = take((size_t)B * Hkv * 4);
  w.pre_ml = take((size_t)w.pre_rows * 8);
  w.pre_o = take((size_t)w.pre_rows * D * 4);
  w.extra_ml = take((size_t)w.extra_rows * 8);
  w.extra_o = take((size_t)w.extra_rows * D * 4);
  w.own_ml = take((size_t)w.own_slots * own_rows * 8);
  w.own_o = take((size_t)w.own_slots * own_rows * D * 4);
  w.total = at;
  return w;
}

struct Args {
  AttentionLaunch a;
  int box;  // tokens of one TMA box, 0: copies by row
  int G, Q, row_tiles, grid;  // heads per key head, K + 1, item tiles of a sequence's rows, CTAs of part_kernel
  uint32_t* head;
  int4* qrow;     // compact query -> b * Q + i, its sequence's drafts, committed tokens and first chunk
  int4* chunk_of;  // chunk -> sequence, its drafts, committed tokens and first chunk
  int* stat;      // a sequence's flags
  int* nan_from;  // [B][Hkv] first own token whose drafted value is not finite
  float2 *pre_ml, *extra_ml, *own_ml;
  float *pre_o, *extra_o, *own_o;
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------------------
// 1. The plan: one CTA, a thread per sequence (up to kPlanThreads).
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kSplits = 256;
// Costs in key tiles of a prefix item (about 1.9 us), fitted to calls measured with other
// plans: the document batch with one part of 128 tiles a prefix item 674 us, with three
// of 43 tiles 706; its prefix alone with three 432, with two 452, with one 531; the 64 x 8
// round with one part of 16 tiles 62, with two of 8 66.
constexpr float kItemTiles = 4.f, kMergeTiles = 4.f, kOwnTiles = 0.8f, kOwnItemTiles = 1.5f;

// Inclusive prefix sum over the CTA (also the total).
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int s = lane < (int)(blockDim.x >> 5) ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return v + (warp > 0 ? before : 0);
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const Args p) {
  __shared__ int warp_sums[32];
  __shared__ unsigned long long tiles2;  // of 2 * kTileKeys keys, all sequences
  __shared__ unsigned flags;
  const AttentionLaunch& a = p.a;
  const int t = threadIdx.x, threads = blockDim.x;  // (whole warps)
  if (t == 0) {
    tiles2 = 0;
    flags = 0;
  }
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  const int step = 2 * kTileKeys;
  // sequence b: its flag, drafts and length (0 tokens if it is flagged)
  auto look = [&](int b, int& k, int& len) {
    k = a.kpr ? a.kpr[b] : a.K;
    len = a.lens[b];
    if (k < 0 || k > a.K) return (int)SV_FLAG_BAD_K;
    if (len < 0 || (long long)len + k > (long long)a.max_pages * a.page_size) return (int)SV_FLAG_BAD_N;
    return 0;
  };
  int k0 = 0, len0 = 0, bad0 = 1;  // this thread's first sequence
  unsigned long long mine = 0;
  for (int b = t; b < a.B; b += threads) {
    int k, len;
    const int bad = look(b, k, len);
    if (b == t) {
      k0 = k;
      len0 = len;
      bad0 = bad;
    }
    p.stat[b] = bad;
    if (bad)
      atomicOr(&flags, (unsigned)bad);
    else
      mine += (unsigned)ceil_div(len + k, step);
  }
  for (long long e = t; e < (long long)a.B * a.Hkv; e += threads) p.nan_from[e] = 0x7fffffff;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if ((t & 31) == 0 && mine) atomicAdd(&tiles2, mine);
  __syncthreads();
  // a chunk: long enough that all chunks together are at most kSlack per CTA beside one per sequence
  const unsigned long long units = tiles2 * (unsigned)(a.Hkv * p.row_tiles), aim = (unsigned long long)kSlack * p.grid;
  int per = 1;  // steps of a chunk
  if (units > aim) per = units < 0xffffffffull ? (int)(((unsigned)units - 1) / (unsigned)aim + 1) : (int)((units - 1) / aim + 1);
  int queries = 0, chunks = 0;
  for (int b0 = 0; b0 < a.B; b0 += threads) {
    const int b = b0 + t;
    int k = k0, len = len0, bad = bad0, q = 0, n = 0;
    if (b0 > 0 && b < a.B) bad = look(b, k, len);
    if (b < a.B && bad == 0) {
      q = k + 1;
      n = ceil_div(ceil_div(len + k, step), per);
    }
    int total;
    const int qe = queries + block_scan(q, warp_sums, total) - q;
    queries += total;
    const int ce = chunks + block_scan(n, warp_sums, total) - n;
    chunks += total;
    for (int i = 0; i < q; ++i) p.qrow[qe + i] = make_int4(b * p.Q + i, k, len, ce);
    for (int c = 0; c < n; ++c) p.chunk_of[ce + c] = make_int4(b, k, len, ce);
  }
  const int ptiles = ceil_div(a.prefix_len, kTileKeys);
  const long long rows = (long long)queries * p.G;
  const int row_items = (int)((rows + kItemRows - 1) / kItemRows) * a.Hkv;
  if (t < 32) {
    // Splits of the prefix, and the CTAs that begin with it: those for which the call is
    // estimated to be done first.  The unit is a key tile of a prefix item; an item's
    // beginning and end cost kItemTiles and its parts in the merge kMergeTiles, 256 keys
    // of a sequence kOwnTiles and an item of them kOwnItemTiles.  CTAs that are done with
    // their list take from the other, so the last item ends with the average of all the
    // work, or with the prefix's rounds where these take longer.  As many CTAs begin with the
    // prefix as end it by then (its items are the longest: begun late they would be the
    // last).  The partial results have room for kSlack * grid items beside one per row item.
    int splits = 0, split_tiles = 0, ctas = 0;
    if (ptiles > 0 && row_items > 0) {
      const float own = kOwnTiles * (float)units + kOwnItemTiles * (float)(chunks * a.Hkv * p.row_tiles);
      const int most = max(1, min(ptiles, kSlack * p.grid / row_items));
      float best = 3e38f;
      for (int c = t + 1; c <= most && c <= kSplits; c += 32) {
        const int tiles = ceil_div(ptiles, c), parts = ceil_div(ptiles, tiles), items = row_items * parts;
        const float item = (float)tiles + kItemTiles, average = ((float)items * item + own) / (float)p.grid;
        const int rounds = max(ceil_div(items, p.grid), min(items, (int)(average / item)));
        const int first = ceil_div(items, rounds);
        const float cost = fmaxf(average, (float)ceil_div(items, first) * item) + (float)items * kMergeTiles / (float)p.grid;
        if (cost < best) {
          best = cost;
          splits = parts;
          split_tiles = tiles;
          ctas = first;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float c = __shfl_xor_sync(0xffffffffu, best, o);
        const int s = __shfl_xor_sync(0xffffffffu, splits, o), n = __shfl_xor_sync(0xffffffffu, split_tiles, o);
        const int f = __shfl_xor_sync(0xffffffffu, ctas, o);
        if (c < best || (c == best && s < splits)) {
          best = c;
          splits = s;
          split_tiles = n;
          ctas = f;
        }
      }
    }
    if (t == 0) {
      p.head[H_PRE_CTAS] = ctas;
      p.head[H_ALL_FAIL] = 0;
      p.head[H_NEXT_PRE] = ctas;  // (these many CTAs take the first ones by themselves)
      p.head[H_NEXT_OWN] = p.grid - ctas;
      p.head[H_QUERIES] = queries;
      p.head[H_CHUNKS] = chunks;
      p.head[H_CHUNK_KEYS] = per * step;
      p.head[H_SPLITS] = splits;
      p.head[H_SPLIT_TILES] = split_tiles;
      p.head[H_PRE_ITEMS] = row_items * splits;
      p.head[H_OWN_ITEMS] = chunks * a.Hkv * p.row_tiles;
      p.head[H_FLAGS] = flags;
    }
  }
}

// ---------------------------------------------------------------------------
// 2. The parts.
// ---------------------------------------------------------------------------
// Warps 0-3, 4-7: softmax of stream 0, 1; 8, 9: their products (one issuing thread
// alone spends as long on its waits and commits as on the products); 10: items and
// Q; 11-15: K and V.
constexpr int kThreads = 512;
constexpr int kSlots = 5;
constexpr int kLoaders = kSlots;  // a warp per slot of the ring: it waits for its own tile's release, never for an older one
// The block is launched with 128 registers a thread; the softmax warps keep a row's
// 128 scores in registers: (176 + 176 + 80 + 80) * 128 = 512 * 128.
constexpr int kSoftmaxRegs = 176, kOtherRegs = 80;
static_assert(2 * (kSoftmaxRegs + kOtherRegs) * 128 <= kThreads * 128, "no more registers than the block was launched with");
constexpr uint32_t kColS = 0, kColO = 256, kStreamCols = 128;

template <int D>
struct Shape {
  static constexpr int kHalves = D / 64;                  // 128-byte columns of a row
  static constexpr int kTileBytes = kTileKeys * D * 2;    // K, V or one stream's Q
  static constexpr int kSmem = 2 * kTileBytes + kSlots * kTileBytes + 1024;
};

struct alignas(16) Item {
  int kind;  // 0 prefix, 1 own, -1 none left
  int h, b;  // key head; sequence (own)
  int row0, rows;    // first row (compact for the prefix, the sequence's for own) and count, at most 256
  int key0, keys;    // first key and number of keys, prefix or own positions
  int tiles;
  int slot;          // split (prefix) or chunk (own)
  int len;           // own: committed tokens
  int unused;
  __device__ __forceinline__ bool pair() const { return rows > 128; }  // streams: two row tiles, or alternate key tiles
  // up to 64 rows stand in Q's tile twice: the second stream uses the copy, whose rows
  // belong to other warps (and schedulers) than the first one's
  __device__ __forceinline__ bool twice() const { return rows <= 64; }
  __device__ __forceinline__ int ahead() const { return pair() ? 1 : 2; }
  __device__ __forceinline__ int stream_tiles(int s) const { return pair() ? tiles : (tiles + 1 - s) / 2; }
};

// Items of this CTA, by one thread: from its preferred list until that is empty, then
// from the other.  Items without keys are passed over.  The first one needs no
// counter: the CTAs that begin with a list take its first items in their order.
struct Feed {
  int list, left;
  int start;  // its place in the order, -1 once that is taken
  int queries, chunk_keys, split_tiles, pre_items, own_items;

  __device__ __forceinline__ void init(const Args& p) {
    const int4* head = reinterpret_cast<const int4*>(p.head);
    const int4 h1 = head[1], h2 = head[2];
    queries = h1.x;
    chunk_keys = h1.z;
    split_tiles = h2.x;
    pre_items = h2.y;
    own_items = h2.z;
    const int ctas = h2.w;
    list = (int)blockIdx.x < ctas ? 0 : 1;
    start = (int)blockIdx.x - (list ? ctas : 0);
    left = 2;
  }
  __device__ __forceinline__ Item decode(const Args& p, int idx) const {
    const AttentionLaunch& a = p.a;
    Item it;
    it.kind = list;
    it.b = it.len = 0;
    if (list == 0) {
      // row tiles fastest: the items in flight share the keys' tiles in L2
      const int row_items = (int)(((long long)queries * p.G + kItemRows - 1) / kItemRows);
      it.row0 = idx % row_items * kItemRows;
      it.h = idx / row_items % a.Hkv;
      it.slot = idx / row_items / a.Hkv;
      const long long left = (long long)queries * p.G - it.row0;
      it.rows = left < kItemRows ? (int)left : kItemRows;
      it.key0 = it.slot * split_tiles * kTileKeys;
      it.keys = min(a.prefix_len - it.key0, split_tiles * kTileKeys);
    } else {
      const int rt = idx % p.row_tiles;
      it.h = idx / p.row_tiles % a.Hkv;
      it.slot = idx / p.row_tiles / a.Hkv;
      const int4 of = p.chunk_of[it.slot];
      it.b = of.x;
      it.len = of.z;
      it.row0 = rt * kItemRows;
      it.rows = min((of.y + 1) * p.G - it.row0, kItemRows);
      it.key0 = (it.slot - of.w) * chunk_keys;
      it.keys = min(it.len + of.y - it.key0, chunk_keys);
      if (it.rows <= 0) it.keys = 0;  // (a sequence with fewer row tiles than the largest)
    }
    it.tiles = it.keys > 0 ? ceil_div(it.keys, kTileKeys) : 0;
    return it;
  }
  __device__ __forceinline__ Item next(const Args& p) {
    Item it;
    while (left > 0) {
      const int i = start >= 0 ? start : (int)atomicAdd(&p.head[list ? H_NEXT_OWN : H_NEXT_PRE], 1u);
      start = -1;
      if (i < (list ? own_items : pre_items)) {
        it = decode(p, i);
        if (it.tiles > 0) return it;
      } else {
        list ^= 1;
        --left;
      }
    }
    it.kind = -1;
    return it;
  }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// bf16 pairs with an exponent of all ones (infinity or NaN)
__device__ __forceinline__ bool not_finite(uint32_t w) {
  return (w & 0x7f800000u) == 0x7f800000u || (w & 0x7f80u) == 0x7f80u;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    part_kernel(const __grid_constant__ Args p, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV) {
  using S = Shape<D>;
  constexpr uint32_t kIdS = tc::idesc(false, false, 128, kTileKeys), kIdO = tc::idesc(false, true, 128, D);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kSlots], raw[kSlots], empty[kSlots], q_full[2], q_empty[2], q_go, s_full[2],
      p_ready[2][2], o_full[2], turn_of[2], item_full[2], item_empty[2], drained[2];
  __shared__ Item items[2];
  __shared__ uint32_t tmem_base;
  __shared__ int2 loaded[kLoaders];  // tiles and looks of a ring slot, at the end
  __shared__ int failed;
  const AttentionLaunch& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t q_smem = smem_addr(smem), ring = q_smem + 2 * S::kTileBytes;
  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], 32);
      mbar_init(&raw[s], 1);
      mbar_init(&empty[s], 2);  // (both streams)
    }
    mbar_init(&q_go, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], 4);  // (four runs of 32 rows)
      mbar_init(&q_empty[s], 2);
      mbar_init(&s_full[s], 1);
      mbar_init(&turn_of[s], 1);
      mbar_init(&p_ready[s][0], 128);
      mbar_init(&p_ready[s][1], 128);
      mbar_init(&o_full[s], 1);
      mbar_init(&drained[s], 1);
      mbar_init(&item_full[s], 1);
      mbar_init(&item_empty[s], 8 + 2 + kLoaders);  // a lane of every other warp
    }
    failed = 0;
    fence_mbar_init();
  }
  if (warp == 8) tc::alloc<1>(&tmem_base, 512);
  if (tid == 9 * 32 && p.box) {
    tc::prefetch_map(&tmK);
    tc::prefetch_map(&tmV);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_base;
  pdl_launch_dependents();
  pdl_wait();

  // The items pass through two slots, written ahead by warp 10.
  auto peek = [&](int n) {  // item n of this CTA, read by a whole warp
    // (word by word: as a structure it would live in local memory)
    const bool ok = __all_sync(
        0xffffffffu, a.wait_tries > 0 && tc::wait_bounded(&item_full[n & 1], (uint32_t)((n >> 1) & 1)));
    if (!ok) failed = 1;
    const int4* from = reinterpret_cast<const int4*>(&items[n & 1]);
    const int4 w0 = from[0], w1 = from[1], w2 = from[2];
    Item got;
    got.kind = ok ? w0.x : -1;
    got.h = w0.y;
    got.b = w0.z;
    got.row0 = w0.w;
    got.rows = w1.x;
    got.key0 = w1.y;
    got.keys = w1.z;
    got.tiles = w1.w;
    got.slot = w2.x;
    got.len = w2.y;
    return got;
  };
  auto fetch = [&](int n) {
    const Item got = peek(n);
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[n & 1]);
    return got;
  };
  auto landed = [&]() {  // this lane's copies, seen by the tensor cores once announced
    asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
    fence_async();
  };
  auto wait = [&](uint64_t* bar, int phase) {
    if (tc::wait_bounded(bar, (uint32_t)(phase & 1))) return true;
    failed = 1;
    return false;
  };

  // An item's Q, by a warp: first + count * 32 rows `stride` runs apart, into the
  // halves of its place from `half` on, once `bar` says that the scores of their last
  // items are done.  A lane finds a row of each run and asks for it in L2, then the
  // warp copies the rows together.  Rows past the end stay as they are: what comes of
  // them is never read.
  // (loops, not straight code: a CTA of short items runs through this once for each of
  // them, and its instructions push the softmax's out of the cache)
  auto load_q = [&](const Item& it, int first, int stride, int end, int half, uint64_t* bar, int phase) {
    constexpr int kWords = D / 8, kRows = 32 / kWords;  // 16-byte words of a row, rows of one instruction
    const int c = lane % kWords, sub = lane / kWords;
    bool ok = true;
#pragma unroll 1
    for (int pass = phase < 0 ? 1 : 0; pass < 2; ++pass) {  // (nothing to wait for: no need to ask ahead)
      if (pass == 1) ok = __all_sync(0xffffffffu, wait(bar, phase));
#pragma unroll 1
      for (int u = first; u < end && ok; u += stride) {
        const int run = (it.twice() ? u & 1 : u) * 32, r = run + lane;
        if (run >= it.rows) continue;  // (the same in the whole warp)
        const uint16_t* line = nullptr;
        if (r < it.rows) {
          const int row = it.row0 + r, qi = row / p.G, g = row - qi * p.G;
          const int bi = it.kind == 0 ? p.qrow[qi].x : it.b * p.Q + qi;
          const int b = bi / p.Q, i = bi - b * p.Q;
          line = static_cast<const uint16_t*>(a.q) + b * a.q_seq + i * a.q_pos + (long long)(it.h * p.G + g) * a.q_head;
        }
        if (pass == 0) {
          if (line) {
            asm volatile("prefetch.global.L2 [%0];" ::"l"(line));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(line + D - 8));
          }
          continue;
        }
        const uint32_t to = q_smem + (half + (u >> 2)) * S::kTileBytes + (c >> 3) * (kTileKeys * 128);
#pragma unroll 2
        for (int v = 0; v < 32 / kRows; ++v) {
          const int rr = (u & 3) * 32 + v * kRows + sub;
          const uint16_t* from =
              reinterpret_cast<const uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(line), v * kRows + sub));
          if (from) cp16(to + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), from + c * 8, true);
        }
      }
    }
    if (!ok) return false;
    landed();
    __syncwarp();
    if (lane == 0)
      for (int u = first; u < end; u += stride) mbar_arrive(&q_full[half + (u >> 2)]);
    return true;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 10) {
      // ---- the items, one ahead, and Q of the items with 128 rows or fewer ----
      Feed feed;
      feed.init(p);
      int q_uses[2] = {0, 0};
      bool ok = true;
      auto publish = [&](int n) {
        if (n >= 2 && !__all_sync(0xffffffffu, wait(&item_empty[n & 1], (n >> 1) - 1))) return false;
        if (lane == 0) {
          items[n & 1] = feed.next(p);
          mbar_arrive(&item_full[n & 1]);
        }
        __syncwarp();
        return true;
      };
      for (int n = 0; ok; ++n) {
        ok = publish(n);
        if (!ok) break;
        const Item it = peek(n);
        if (it.kind < 0) break;
        if (it.pair()) {  // the ring's warps load it
          ok = __all_sync(0xffffffffu, wait(&q_empty[0], q_uses[0]++ - 1) && wait(&q_empty[1], q_uses[1]++ - 1));
          if (ok && lane == 0) mbar_arrive(&q_go);
        } else {
          ok = load_q(it, 0, 1, 4, n & 1, &q_empty[n & 1], q_uses[n & 1] - 1);
          ++q_uses[n & 1];
        }
      }
    } else if (warp > 10) {
      // ---- K and V: a warp per slot of the ring ----
      const int slot = warp - 11;
      int turn = 0, use = 0, looks = 0;  // tiles of all slots before this item; of this one; of those looked at
      int pairs = 0;  // items of two row tiles so far
      bool ok = true;
      constexpr int kWords = D / 8, kRows = 32 / kWords;
      const int c = lane % kWords, sub = lane / kWords;
      const uint32_t base = ring + slot * S::kTileBytes + (c >> 3) * (kTileKeys * 128);
      for (int n = 0; ok; ++n) {
        const Item it = fetch(n);
        if (it.kind < 0) break;
        // K_0 .. K_{d-1}, then V_j, K_{j+d}
        const int d = it.ahead() < it.tiles ? it.ahead() : it.tiles;
        const int total = 2 * it.tiles;
        bool q_due = it.pair();  // two row tiles: Q is loaded by these warps, behind their first tile
        auto my_q = [&]() {
          q_due = false;
          ok = load_q(it, slot, kSlots, 8, 0, &q_go, pairs);
          ++pairs;
        };
        for (int x = (slot + kSlots - turn % kSlots) % kSlots; x < total; x += kSlots) {
          // which tile: x < d: K_x; else pairs (V_j, K_{j+d}) while both exist, then the last V's
          int j = x, is_v = 0;
          if (x >= d) {
            const int y = x - d, both = 2 * (it.tiles - d);
            is_v = y >= both || (y & 1) == 0;
            j = y >= both ? (it.tiles - d) + (y - both) : (is_v ? y >> 1 : (y >> 1) + d);
          }
          const int first = it.key0 + j * kTileKeys, keys_left = it.keys - j * kTileKeys;
          const int end = keys_left < kTileKeys ? keys_left : kTileKeys;
          int drafted = it.kind == 1 && is_v ? it.len - first : kTileKeys;  // first row of a drafted token's value
          if (drafted < 0) drafted = 0;
          auto page_of = [&](int key, int& off) {  // the page's id, -1 if it is not one
            const int pg = key / a.page_size;
            off = key - pg * a.page_size;
            const int id = it.kind == 0 ? a.prefix_pages[pg] : a.table[(long long)it.b * a.max_pages + pg];
            if ((unsigned)id < (unsigned)a.num_pages) return id;
            if (it.kind == 0)
              p.head[H_ALL_FAIL] = 1;
            else
              atomicOr(&p.stat[it.b], SV_FLAG_BAD_PAGE);
            atomicOr(&p.head[H_FLAGS], SV_FLAG_BAD_PAGE);
            return -1;
          };
          // rows of V to be looked at once they have landed: drafted tokens', and those
          // past the end, which a box brings along
          const bool look = drafted < end || (p.box && is_v && end < kTileKeys);
          if (p.box) {
            // a lane per box: 64 columns of p.box tokens
            const int at = lane / S::kHalves * p.box, half = lane % S::kHalves;
            int off = 0, id = -1;
            if (at < end) id = page_of(first + at, off);
            if (use > 0) ok = __all_sync(0xffffffffu, wait(&empty[slot], use - 1));
            if (!ok) break;
            const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, id >= 0)) * p.box * 128);
            uint64_t* bar = look ? &raw[slot] : &full[slot];
            if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (id >= 0)
              tc::tma_load_4d(ring + slot * S::kTileBytes + half * (kTileKeys * 128) + at * 128, is_v ? &tmV : &tmK,
                              half * 64, off, it.h, id, bar);
            if (look) {
              ok = __all_sync(0xffffffffu, wait(&raw[slot], looks++));
              if (!ok) break;
              for (int r = end + sub; r < kTileKeys; r += kRows)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                 base + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                             "r"(0)
                             : "memory");
              fence_async();
            } else if (lane != 0) {
              mbar_arrive(&full[slot]);
            }
          } else {
            const uint16_t* pool = static_cast<const uint16_t*>(is_v ? a.v : a.k) + it.h * a.head + c * 8;
            // this lane finds the places of rows lane, lane + 32, ...
            long long at[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              at[u] = -1;
              int off;
              if (u * 32 + lane < end) {
                const int id = page_of(first + u * 32 + lane, off);
                if (id >= 0) at[u] = id * a.page + off * a.token;
              }
            }
            if (use > 0) ok = __all_sync(0xffffffffu, wait(&empty[slot], use - 1));
            if (!ok) break;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll 4
              for (int v = 0; v < 32 / kRows; ++v) {
                const int r = u * 32 + v * kRows + sub;
                const long long from = __shfl_sync(0xffffffffu, at[u], v * kRows + sub);
                cp16(base + r * 128 + (((c & 7) ^ (r & 7)) << 4), pool + (from < 0 ? 0 : from), from >= 0);
              }
            landed();
          }
          // Values of drafted tokens: positions in front of one have weight 0 there, and
          // 0 times a value that is not finite would reach their sums.  Such words
          // become zeros; the merge fails the positions that do see them.
          if (drafted < end) {
            __syncwarp();
#pragma unroll 1
            for (int r = drafted + sub; r < end; r += kRows) {
              const uint32_t at_s = base + r * 128 + (((c & 7) ^ (r & 7)) << 4);
              uint4 q;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                           : "r"(at_s)
                           : "memory");
              if (not_finite(q.x) || not_finite(q.y) || not_finite(q.z) || not_finite(q.w)) {
                atomicMin(&p.nan_from[(long long)it.b * a.Hkv + it.h], first + r);
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at_s), "r"(0) : "memory");
              }
            }
            fence_async();
          }
          if (look || !p.box) mbar_arrive(&full[slot]);
          ++use;
          if (q_due && ok) my_q();
          if (!ok) break;
        }
        if (!ok) break;
        if (q_due) my_q();
        turn += total;
      }
      if (lane == 0) loaded[slot] = make_int2(use, looks);
    } else {
      // ---- the products of one stream, issued by one thread ----
      const int s = warp - 8;
      uint32_t slot = 0, phase = 0;  // the ring's next tile
      uint32_t p_phase = 0, next_phase = 0, q_phase[2] = {0, 0};
      bool opening = s == 0;  // the first turn of all, which no other precedes
      const uint32_t ring_lo = tc::desc_low(ring, kTileKeys * 128);
      const uint32_t col_s = tmem + kColS + s * kStreamCols, col_o = tmem + kColO + s * kStreamCols;
      for (int n = 0;; ++n) {
        const Item it = fetch(n);
        if (it.kind < 0) break;
        bool ok = true;
        if (lane == 0) {
          const int T = it.tiles, d = it.ahead() < T ? it.ahead() : T;
          const bool pr = it.pair();
          const int mine = pr ? s : n & 1;  // half of Q's place
          const uint32_t q_lo = tc::desc_low(q_smem, 16) + mine * (S::kTileBytes >> 4);
          struct Tile {
            uint32_t lo;
            uint64_t* empty;
          };
          auto take = [&]() {  // the next tile, once it has landed
            if (ok) ok = wait(&full[slot], (int)phase);
            const Tile t = {ring_lo + slot * (S::kTileBytes >> 4), &empty[slot]};
            if (++slot == kSlots) {
              slot = 0;
              phase ^= 1;
            }
            return t;
          };
          auto scores = [&](const Tile& k) {  // S = Q K^T
            tc::fence_after();
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
              const uint32_t off = (q >> 2) * (kTileKeys * 128 >> 4) + (q & 3) * 2;
              tc::mma_low(col_s, q_lo + off, k.lo + off, kIdS, q != 0);
            }
            tc::commit<1>(smem_addr(&s_full[s]));
          };
          // O += P V, half of the keys as soon as their weights are there.  Two row tiles
          // take turns with their products: left alone they fall into step, both in
          // their softmax at the same time and then both at the tensor cores (3900
          // clocks a tile, 2048 of them products)
          auto values = [&](const Tile& v, bool acc, bool in_turn) {
#pragma unroll
            for (int q = 0; q < kTileKeys / 16; ++q) {
              if (q % (kTileKeys / 32) == 0) {
                if (ok) ok = wait(&p_ready[s][q / (kTileKeys / 32)], (int)p_phase);
                if (q == 0 && in_turn) {
                  if (ok) ok = wait(&turn_of[s], (int)next_phase);
                  next_phase ^= 1;
                }
                tc::fence_after();
              }
              tc::mma_ts_low(col_o, col_s + 8 * q, v.lo + q * (2048 >> 4), kIdO, acc || q != 0);
            }
            p_phase ^= 1;
          };
          // both streams wait for every tile and every half of Q in use, and release
          // them once each: a release can so never count for an earlier use
          for (int h = pr ? 0 : mine; h <= (pr ? 1 : mine) && ok; ++h) {
            ok = wait(&q_full[h], (int)q_phase[h]);
            q_phase[h] ^= 1;
          }
          int left = it.stream_tiles(s);  // scores to come
          auto scored = [&](const Tile& k) {  // (its slot and Q's, behind its scores)
            tc::commit<1>(smem_addr(k.empty));
            if (--left == 0) tc::commit<1>(smem_addr(&q_empty[mine]));
          };
          if (ok && pr) mbar_arrive(&q_empty[s ^ 1]);
          if (ok && left == 0) mbar_arrive(&q_empty[mine]);
          for (int x = 0; x < d && ok; ++x) {
            const Tile k = take();
            if (!ok) break;
            if (pr || x == s) {
              scores(k);
              scored(k);
            } else {
              mbar_arrive(k.empty);
            }
          }
          for (int j = 0; j < T && ok; ++j) {
            // O += P(j) V_j, then the next scores over P's place (the products of one
            // thread run in order)
            const Tile v = take();
            if (!ok) break;
            const bool own = pr || (j & 1) == s, more = j + d < T;
            Tile k;
            if (more) k = take();
            if (!ok) break;
            if (own) {
              values(v, pr ? j > 0 : j > 1, pr && !opening);
              if (pr) opening = false;
              if (!ok) break;
              if (!pr) tc::commit<1>(smem_addr(v.empty));
              if (more)
                scores(k);
              else
                tc::commit<1>(smem_addr(&o_full[s]));
              if (pr) {  // the other's turn before the release: each commit holds this thread up
                mbar_arrive(&turn_of[s ^ 1]);
                tc::commit<1>(smem_addr(v.empty));
              }
              if (more) scored(k);
            } else {
              mbar_arrive(v.empty);
              if (more) mbar_arrive(k.empty);
            }
          }
        }
        if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax of one stream: a row per thread ----
    const int s = warp >> 2, row = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t col_s = lanes + kColS + s * kStreamCols, col_o = lanes + kColO + s * kStreamCols;
    // (a scale of 0 as one too small to be seen: a masked score of -inf then still has weight 0)
    const float c = a.scale == 0.f ? 1e-30f : a.scale * kLog2e;
    const float worst = c >= 0.f ? -INFINITY : INFINITY;
    int s_turn = 0, o_turn = 0;
    bool ok = true;
    Item it = fetch(0);
    for (int n = 1; it.kind >= 0; ++n) {
      const int tiles = it.stream_tiles(s);
      if (tiles == 0) {
        it = fetch(n);
        continue;
      }
      // this thread's row, of the item and among all
      const int mine = it.pair() ? s * 128 + row : (it.twice() ? row - 64 * s : row), r = it.row0 + mine;
      const bool live = mine >= 0 && mine < it.rows;
      const bool warp_live = __any_sync(0xffffffffu, live);
      // keys that the row sees, from the item's first on
      int sees = 0;
      if (live) sees = it.kind == 0 ? it.keys : min(it.keys, it.len + r / p.G - it.key0);
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < tiles; ++j) {
        const int first = (it.pair() ? j : 2 * j + s) * kTileKeys;
        const int vis = max(0, min(kTileKeys, sees - first));
        if (!__all_sync(0xffffffffu, wait(&s_full[s], s_turn))) {
          ok = false;
          break;
        }
        ++s_turn;
        if (!warp_live) {  // rows that nothing is read from: any weights will do
          mbar_arrive(&p_ready[s][0]);
          mbar_arrive(&p_ready[s][1]);
          continue;
        }
        tc::fence_after();
        const bool all = __all_sync(0xffffffffu, vis == kTileKeys);
        // the row's scores, and their extreme
        uint32_t v[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tc::ld32(col_s + 32 * q, v[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q) tc::ld_wait(v[q]);
        if (!all) {
#pragma unroll
          for (int e = 0; e < kTileKeys; ++e)
            if (e >= vis) v[e >> 5][e & 31] = __float_as_uint(worst);
        }
        float top;
        {
          float t[4] = {worst, worst, worst, worst};
          if (c >= 0.f) {
#pragma unroll
            for (int e = 0; e < kTileKeys; e += 2)
              t[e / 2 & 3] = max3(t[e / 2 & 3], __uint_as_float(v[e >> 5][e & 31]), __uint_as_float(v[e >> 5][(e & 31) + 1]));
            top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
          } else {
#pragma unroll
            for (int e = 0; e < kTileKeys; ++e) t[e & 3] = fminf(t[e & 3], __uint_as_float(v[e >> 5][e & 31]));
            top = fminf(fminf(t[0], t[1]), fminf(t[2], t[3]));
          }
        }
        // Weights are taken relative to a reference that follows the maximum only
        // when that is 2^8 above it: float32 sums and bf16 weights lose nothing by
        // it, and the accumulator is hardly ever rescaled.
        const float mt = vis > 0 && top != worst ? top * c : -INFINITY;
        const bool raise = mt > m + 8.f || (m == -INFINITY && mt > -INFINITY);
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? (m == -INFINITY ? 0.f : ex2(m - mt)) : 1.f;
          if (raise) m = mt;
          l *= f;
          if (j > 0) {  // (the product before this tile's scores is complete, too)
#pragma unroll 1
            for (int q = 0; q < D; q += 16) {
              uint32_t o[16];
              tc::ld16(col_o + q, o);
              tc::ld_wait(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tc::st16(col_o + q, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const F2 c2 = f2_pack(c, c), ref2 = f2_pack(-ref, -ref);
        F2 sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x, y;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(v[q][e]), __uint_as_float(v[q][e + 1])), c2, ref2), x, y);
            x = ex2(x);
            y = ex2(y);
            sum[e / 2 & 1] = f2_add(sum[e / 2 & 1], f2_pack(x, y));
            w[e >> 1] = tc::pack_bf16x2(x, y);
          }
          tc::st16(col_s + 16 * q, w);  // over scores that this thread has read
          if (q & 1) {
            tc::st_wait();
            tc::fence_before();
            mbar_arrive(&p_ready[s][q >> 1]);
          }
        }
        float a0, a1, b0, b1;
        f2_unpack(sum[0], a0, a1);
        f2_unpack(sum[1], b0, b1);
        l += (a0 + a1) + (b0 + b1);
      }
      if (!ok) break;
      ok = __all_sync(0xffffffffu, wait(&o_full[s], o_turn));
      ++o_turn;
      if (!ok) break;
      tc::fence_after();
      // (the next item before the stores: the release of its place would wait for them)
      const Item next = fetch(n);
      // this row's part, in quads of columns: [D / 4][rows][4], so that a warp's 32 rows
      // are 512 contiguous bytes of a store and not 32 lines
      long long at, rows_o;
      float2* ml;
      float* o;
      if (it.kind == 0) {
        const int queries = p.head[H_QUERIES];
        if (s == 1 && !it.pair()) {
          rows_o = 128;
          at = (long long)it.slot * a.Hkv + it.h;
          ml = p.extra_ml + at * rows_o + mine;
          o = p.extra_o + at * rows_o * D + mine * 4;
        } else {
          rows_o = (long long)queries * p.G;
          at = (long long)it.slot * a.Hkv + it.h;
          ml = p.pre_ml + at * rows_o + r;
          o = p.pre_o + at * rows_o * D + r * 4;
        }
      } else {
        rows_o = p.Q * p.G;
        at = ((long long)it.slot * a.Hkv + it.h) * 2 + (it.pair() ? 0 : s);
        ml = p.own_ml + at * rows_o + r;
        o = p.own_o + at * rows_o * D + r * 4;
      }
      if (live) *ml = make_float2(m, l);
#pragma unroll 1
      for (int q = 0; q < D && warp_live; q += 16) {
        uint32_t v[16];
        tc::ld16(col_o + q, v);
        tc::ld_wait(v);
        if (live) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(o + (q / 4 + e) * rows_o * 4) =
                make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
      }
      tc::fence_before();  // (the next item's first weights follow: its product may overwrite O)
      it = next;
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (failed) {  // (the same in every thread) a wait ran out: copies and products on their way end first
    if (lane == 0 && (warp == 8 || warp == 9)) {
      tc::commit<1>(smem_addr(&drained[warp - 8]));
      (void)tc::wait_bounded(&drained[warp - 8], 0);
    }
    if (lane == 0 && warp > 10) {
      const int slot = warp - 11, use = loaded[slot].x, looks = loaded[slot].y;
      if (looks > 0) (void)tc::wait_bounded(&raw[slot], (uint32_t)((looks - 1) & 1));
      if (use > 0) (void)tc::wait_bounded(&full[slot], (uint32_t)((use - 1) & 1));
    }
    if (tid == 0) {  // parts are missing, and which ones is not known
      p.head[H_ALL_FAIL] = 1;
      atomicOr(&p.head[H_FLAGS], SV_FLAG_TIMEOUT);
    }
    __syncthreads();
  }
  if (warp == 8) tc::dealloc<1>(tmem, 512);
}

// ---------------------------------------------------------------------------
// 3. The parts of a row together.  A warp has eight rows and four quads of columns
// of each (eight rows' quads are a whole line); kGroups warps share the rows.  Small
// calls are bound by the chain of loads that depend on each other (what a row is, its
// parts): one word has all of a row, and kAtOnce parts come with their maxima and sums
// under a running maximum (one token 17.5 -> 15.7 us, 64 x 8 round 62.8 -> 61.2, 33
// sequences of 12 heads 35.6 -> 32.0, against maxima first and one more load of each).
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const Args p) {
  const AttentionLaunch& a = p.a;
  constexpr int N = 2, kGroups = D / 16 / N;  // quads of a thread, warps per eight rows
  constexpr int kAtOnce = 3;  // (2 and 4: 33.0 and 32.1 us in the last of these, 16.9 and 16.3 in the first)
  const float nan = __int_as_float(0x7fffffff);
  pdl_wait();
  const int lane = threadIdx.x & 31, sub = lane & 3;
  const unsigned wid = blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
  const int queries = p.head[H_QUERIES], group = (int)(wid % kGroups);
  const unsigned rows = (unsigned)queries * p.G, id = wid / kGroups * 8 + (lane >> 2);

  if (p.head[H_FLAGS] & (SV_FLAG_BAD_K | SV_FLAG_BAD_N)) {
    // sequences that have no rows: every position that the caller reads is NaN
    for (long long b = blockIdx.x; b < a.B; b += gridDim.x) {
      const int bad = p.stat[b];
      if (!(bad & (SV_FLAG_BAD_K | SV_FLAG_BAD_N))) continue;
      const int n = bad & SV_FLAG_BAD_K ? p.Q : (a.kpr ? a.kpr[b] : a.K) + 1;
      const long long heads = (long long)n * a.Hq;  // (times D: past 2^31)
      for (long long e = threadIdx.x; e < heads * D; e += kMergeThreads) {
        const int row = (int)(e / D), d = (int)(e % D), i = row / a.Hq, h = row - i * a.Hq;
        static_cast<uint16_t*>(a.out)[b * a.o_seq + i * a.o_pos + h * a.o_head + d] = 0x7fff;
        if (a.lse && d == 0) a.lse[(b * p.Q + i) * a.Hq + h] = nan;
      }
    }
  }
  if (rows == 0 || id >= rows * a.Hkv) return;
  const int h = (int)(id / rows);
  const unsigned r = id - h * rows, query = r / p.G;
  const int g = (int)(r - query * p.G);
  const int4 of = p.qrow[query];
  const int bi = of.x, k = of.y, len = of.z, first = of.w;
  const int b = bi / p.Q, i = bi - b * p.Q, hq = h * p.G + g;
  const int splits = p.head[H_SPLITS], per = p.head[H_SPLIT_TILES], keys = p.head[H_CHUNK_KEYS];
  const bool dead = p.stat[b] || p.head[H_ALL_FAIL];
  const bool lost = len + i > p.nan_from[(long long)b * a.Hkv + h];

  // The row's parts: of the prefix, `extra` ones of second streams there (the last split
  // has none if it is a single tile), and the chunks', of one stream or two.
  const unsigned tile0 = r / kItemRows * kItemRows;
  const int ptiles = ceil_div(a.prefix_len, kTileKeys), own = i * p.G + g, all = p.Q * p.G, chunks = ceil_div(len + k, keys);
  const int extra = rows - tile0 > 128 || per < 2 ? 0 : splits - (ptiles - (splits - 1) * per < 2 ? 1 : 0);
  const bool two = (k + 1) * p.G - own / kItemRows * kItemRows <= 128;
  const int before = splits + extra, last = len + k - (chunks - 1) * keys;
  const int parts = dead ? 0 : before + (two ? 2 * chunks - (last > kTileKeys ? 0 : 1) : chunks);
  const int quad = (group * N * 4 + sub) * 4;
  float M = -INFINITY, l = 0.f, acc[N][4];
#pragma unroll
  for (int q = 0; q < N; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[q][e] = 0.f;
  for (int n = 0; n < parts; n += kAtOnce) {
    // kAtOnce parts' loads in flight together
    float2 x[kAtOnce];
    float4 v[kAtOnce][N];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int at = n + u;
      x[u] = make_float2(-INFINITY, 0.f);
      if (at >= parts) continue;
      const float2* ml;
      const float* o;
      long long rows_o;
      if (at < before) {
        const bool second = at >= splits;
        const long long part = (long long)(second ? at - splits : at) * a.Hkv + h;
        rows_o = second ? 128 : rows;
        const unsigned row = second ? r - tile0 : r;
        ml = (second ? p.extra_ml : p.pre_ml) + part * rows_o + row;
        o = (second ? p.extra_o : p.pre_o) + part * rows_o * D + row * 4;
      } else {
        const int c = two ? at - before : 2 * (at - before);
        const long long part = ((long long)(first + (c >> 1)) * a.Hkv + h) * 2 + (c & 1);
        rows_o = all;
        ml = p.own_ml + part * rows_o + own;
        o = p.own_o + part * rows_o * D + own * 4;
      }
      x[u] = *ml;
#pragma unroll
      for (int q = 0; q < N; ++q) v[u][q] = *reinterpret_cast<const float4*>(o + (quad + q * 16) * rows_o);
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) top = x[u].x > top ? x[u].x : top;
    const float f = M == top ? 1.f : ex2(M - top);
    M = top;
    l *= f;
#pragma unroll
    for (int q = 0; q < N; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[q][e] *= f;
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      // a part that saw nothing has weight 0, whatever is there (a NaN in its sum goes on)
      const float w = x[u].x == -INFINITY ? (x[u].y == 0.f ? 0.f : 1.f) : ex2(x[u].x - M);
      l += x[u].y * w;
      if (w == 0.f) continue;
#pragma unroll
      for (int q = 0; q < N; ++q) {
        acc[q][0] = __fmaf_rn(v[u][q].x, w, acc[q][0]);
        acc[q][1] = __fmaf_rn(v[u][q].y, w, acc[q][1]);
        acc[q][2] = __fmaf_rn(v[u][q].z, w, acc[q][2]);
        acc[q][3] = __fmaf_rn(v[u][q].w, w, acc[q][3]);
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* op = static_cast<uint16_t*>(a.out) + b * a.o_seq + i * a.o_pos + hq * a.o_head + quad;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    uint2 w = make_uint2(0x7fff7fffu, 0x7fff7fffu);
    if (!dead && !lost)
      w = make_uint2(tc::pack_bf16x2(acc[q][0] * inv, acc[q][1] * inv), tc::pack_bf16x2(acc[q][2] * inv, acc[q][3] * inv));
    *reinterpret_cast<uint2*>(op + q * 16) = w;
  }
  if (a.lse && sub == 0 && group == 0)
    a.lse[(long long)bi * a.Hq + hq] = dead ? nan : (l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2);
}

template <typename... A>
static cudaError_t launch(void (*k)(A...), unsigned grid, unsigned threads, size_t smem, cudaStream_t st, const A&... p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p...);
}

template <int D>
static cudaError_t run(const Args& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  static std::atomic<int> ready[kMaxDevices];
  const int d = current_device();
  if (d < 0) return cudaErrorInvalidDevice;
  if (!ready[d].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(part_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::kSmem);
    if (e != cudaSuccess) return e;
    ready[d].store(1, std::memory_order_release);
  }
  const int threads = p.a.B < kPlanThreads ? (p.a.B + 31) / 32 * 32 : kPlanThreads;
  cudaError_t e = launch(plan_kernel, 1, (unsigned)threads, 0, st, p);
  if (e == cudaSuccess) e = launch(part_kernel<D>, (unsigned)p.grid, kThreads, Shape<D>::kSmem, st, p, k, v);
  const long long rows = (long long)p.a.B * p.Q * p.a.Hq;
  if (e == cudaSuccess)
    e = launch(merge_kernel<D>, (unsigned)((((rows + 7) / 8) * (D / 32) * 32 + kMergeThreads - 1) / kMergeThreads), kMergeThreads,
               0, st, p);
  return e;
}

// The pool as a 4-D tensor map: 64 of D, `box` tokens of a page, key head, page.
static bool pool_map(tc::EncodeTiledFn enc, CUtensorMap* map, const void* pool, const AttentionLaunch& a, int box) {
  const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.page_size, (cuuint64_t)a.Hkv, (cuuint64_t)a.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)a.token * 2, (cuuint64_t)a.head * 2, (cuuint64_t)a.page * 2};
  const cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1}, estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool), dims, strides, boxes, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace att

size_t attention_workspace_bytes(int B, int K, int Hq, int Hkv, int D, int prefix_len, int max_own) {
  return att::layout(B, K, Hq, Hkv, D, prefix_len, max_own).total;
}

int attention_launch(const AttentionLaunch& L, std::string* err) {
  att::Args p;
  p.a = L;
  p.G = L.Hq / L.Hkv;
  p.Q = L.K + 1;
  p.row_tiles = (p.Q * p.G + att::kItemRows - 1) / att::kItemRows;
  const int sms = tc::num_sms();
  p.grid = sms < att::kMaxGrid ? sms : att::kMaxGrid;
  const att::Layout w = att::layout(L.B, L.K, L.Hq, L.Hkv, L.D, L.prefix_len, (long long)L.max_pages * L.page_size);
  char* base = static_cast<char*>(L.workspace);
  p.head = reinterpret_cast<uint32_t*>(base);
  p.qrow = reinterpret_cast<int4*>(base + w.qrow);
  p.chunk_of = reinterpret_cast<int4*>(base + w.chunk_of);
  p.stat = reinterpret_cast<int*>(base + w.stat);
  p.nan_from = reinterpret_cast<int*>(base + w.nan_from);
  p.pre_ml = reinterpret_cast<float2*>(base + w.pre_ml);
  p.pre_o = reinterpret_cast<float*>(base + w.pre_o);
  p.extra_ml = reinterpret_cast<float2*>(base + w.extra_ml);
  p.extra_o = reinterpret_cast<float*>(base + w.extra_o);
  p.own_ml = reinterpret_cast<float2*>(base + w.own_ml);
  p.own_o = reinterpret_cast<float*>(base + w.own_o);
  cudaStream_t st = static_cast<cudaStream_t>(L.stream);
  // TMA boxes hold whole eights of rows (the swizzle's period) and divide a tile
  CUtensorMap k = {}, v = {};
  p.box = 0;
  if (L.page_size >= 8 && (L.page_size & (L.page_size - 1)) == 0) {
    tc::EncodeTiledFn enc = tc::encoder(err);
    if (!enc) return SV_ERR_CUDA;
    const int box = L.page_size < att::kTileKeys ? L.page_size : att::kTileKeys;
    if (att::pool_map(enc, &k, L.k, L, box) && att::pool_map(enc, &v, L.v, L, box)) p.box = box;
  }
  const cudaError_t e = L.D == 128 ? att::run<128>(p, k, v, st) : att::run<64>(p, k, v, st);
  if (e != cudaSuccess) {
    *err = std::string("attention launch: ") + cudaGetErrorString(e);
    return SV_ERR_CUDA;
  }
  return SV_OK;
}

}  // namespace sv
