// Moves of a paged cache's pages: copies, forks of sequences, the release of
// ended ones, and the compaction of a pool.  They extend the page-granular
// rollback of "Self-speculative decoding with layer skip and KV reuse" §3.3,
// §4.5 to pages that several sequences own: shares[p] counts a page's owners
// beyond the first, so that a page of one sequence (every page that the commit
// gives back, since a fork copies the page that is partly full) has 0.
//
// Which page goes where is decided by ranks (of a fork among the forks that copy,
// of an id among the free or the live ones), never by the order of atomics: the
// same inputs give the same ids.  The copies are bound by memory: a warp takes 2 KB
// of a page at a time, four 16-byte words a lane in flight, and every page array
// has its own row of the grid.  64 forks over 64 arrays of 32 KB pages: 24 to 27 us,
// 252 MB in and out, partly through L2 (37 us at the measured copy rate); a pool of
// 4096 pages of which 2048 move half: 21 us for the copies (19.8 us by their bytes).
// The plans are single kernels of a few us before them.
#include <cstdint>

#include "sv_tc.cuh"

namespace sv {
namespace pages {

constexpr int kThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kFew = 8;  // page arrays of the short argument list (the long one is 4 KB)
constexpr uint32_t kFull = 0xffffffffu;

// Workspace: words 0 flags, 1 moves, 2 the free stack's top or the live pages; then the lists.
constexpr int kHead = 64;

template <int N>
struct Pools {
  uint8_t* base[N];
  long long bytes[N];
};
template <int N>
Pools<N> pools_of(const PagePools& p) {
  Pools<N> r = {};
  for (int i = 0; i < p.n; ++i) {
    r.base[i] = p.base[i];
    r.bytes[i] = p.bytes[i];
  }
  return r;
}

// This CTA's part of the copies of one page array: pairs (src[i], dst[i]), i < n.
__device__ __forceinline__ void copy_pages(uint8_t* base, long long bytes, const int32_t* src, const int32_t* dst, int n,
                                           int num_pages, uint32_t* flags) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 31;
  const int words = (int)(bytes / 16);
  const int pieces = (words + 32 * U - 1) / (32 * U);
  const long long units = (long long)n * pieces;
  for (long long u = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units;
       u += (long long)gridDim.x * (kThreads / 32)) {
    const int m = (int)(u / pieces), w0 = (int)(u - (long long)m * pieces) * 32 * U + lane;
    const int from = src[m], to = dst[m];
    if (from < 0 || from >= num_pages || to < 0 || to >= num_pages) {
      if (lane == 0) atomicOr(flags, SV_FLAG_BAD_PAGE);
      continue;
    }
    if (from == to) continue;
    const uint4* s = reinterpret_cast<const uint4*>(base + from * bytes);
    uint4* d = reinterpret_cast<uint4*>(base + to * bytes);
    uint4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (w0 + 32 * k < words) v[k] = __ldcs(s + w0 + 32 * k);
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (w0 + 32 * k < words) __stcs(d + w0 + 32 * k, v[k]);
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    copy_kernel(const __grid_constant__ Pools<N> p, int num_pages, const int32_t* src, const int32_t* dst, int n,
                uint32_t* ws) {
  pdl_launch_dependents();
  pdl_wait();
  copy_pages(p.base[blockIdx.y], p.bytes[blockIdx.y], src, dst, n, num_pages, ws);
}

// ---------------------------------------------------------------------------
// Forks
// ---------------------------------------------------------------------------
struct ForkArgs {
  int num_pages, page_size, max_pages, F, B;
  int32_t* table;
  int32_t* lens;
  int32_t* shares;
  const int32_t* stack;
  int32_t* top;
  const int32_t* src;
  const int32_t* dst;
  uint32_t* ws;
  int32_t* last;  // [F]: the page to copy, -1 for none, -2 for a fork that is refused
};

// A warp per fork: is it sound, and does it copy a page?
__global__ void __launch_bounds__(kThreads) fork_check_kernel(const ForkArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int f = (int)((blockIdx.x * (long long)kThreads + threadIdx.x) >> 5);
  if (f == 0 && lane == 0) a.ws[2] = (uint32_t)*a.top;
  if (f >= a.F) return;  // (whole warps)
  const int s = a.src[f], d = a.dst[f];
  bool ok = s >= 0 && s < a.B && d >= 0 && d < a.B && s != d;
  // a row that is forked into must not be forked from, nor into twice
  for (int j = lane; j < a.F; j += 32) {
    const int other = a.dst[j];
    if (other == s || (j != f && (other == d || a.src[j] == d))) ok = false;
  }
  ok = __all_sync(kFull, ok);
  uint32_t flag = ok ? 0 : SV_FLAG_BAD_N;
  int last = -1;
  if (ok) {
    const int L = a.lens[s];
    if (L < 0 || (long long)L > (long long)a.max_pages * a.page_size || a.lens[d] != 0) {
      flag = SV_FLAG_BAD_N;
    } else {
      const int full = L / a.page_size, used = full + (L > full * a.page_size);
      const int32_t* from = a.table + (long long)s * a.max_pages;
      const int32_t* to = a.table + (long long)d * a.max_pages;
      bool empty = true, sound = true;
      for (int j = lane; j < a.max_pages; j += 32) {
        empty = empty && to[j] < 0;
        if (j < used) sound = sound && from[j] >= 0 && from[j] < a.num_pages;
      }
      if (!__all_sync(kFull, empty)) flag = SV_FLAG_BAD_N;
      else if (!__all_sync(kFull, sound)) flag = SV_FLAG_BAD_PAGE;
      else if (used > full) last = from[full];
    }
  }
  if (lane == 0) {
    if (flag) atomicOr(a.ws, flag);
    a.last[f] = flag ? -2 : last;
  }
}

// Every CTA ranks the forks that copy (the fork of rank r takes the r-th page from the top of
// the stack); the warps of the first row of the grid write the tables, all copy.
template <int N>
__global__ void __launch_bounds__(kThreads) fork_apply_kernel(const __grid_constant__ Pools<N> p, const ForkArgs a) {
  __shared__ int32_t from[kMaxForks], to[kMaxForks];
  __shared__ int warp_sum[kThreads / 32];
  __shared__ int unsound;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (a.F + kThreads - 1) / kThreads;
  if (tid == 0) unsound = 0;
  int mine = 0;
  for (int j = tid * each; j < min(a.F, (tid + 1) * each); ++j) mine += a.last[j] >= 0;
  int up = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int v = __shfl_up_sync(kFull, up, m);
    if (lane >= m) up += v;
  }
  if (lane == 31) warp_sum[warp] = up;
  __syncthreads();
  int rank = up - mine, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) rank += warp_sum[w];
    total += warp_sum[w];
  }
  const int top = (int)a.ws[2];
  if (top < 0 || top > a.num_pages || total > top) {  // (the same test in every thread)
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) atomicOr(a.ws, SV_FLAG_CAPACITY);
    return;
  }
  for (int j = tid * each; j < min(a.F, (tid + 1) * each); ++j) {
    const int page = a.last[j];
    if (page >= 0) {
      const int fresh = a.stack[top - 1 - rank];
      if (fresh < 0 || fresh >= a.num_pages) unsound = 1;
      from[rank] = page;
      to[rank] = fresh;
      ++rank;
    }
  }
  __syncthreads();
  if (unsound) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) atomicOr(a.ws, SV_FLAG_BAD_PAGE);
    return;
  }
  if (blockIdx.y == 0) {
    if (blockIdx.x == 0 && tid == 0) *a.top = top - total;
    for (int f = blockIdx.x * (kThreads / 32) + warp; f < a.F; f += gridDim.x * (kThreads / 32)) {
      const int page = a.last[f];
      if (page < -1) continue;
      const int s = a.src[f], d = a.dst[f], L = a.lens[s], full = L / a.page_size;
      int before = 0;  // forks in front that copy
      for (int j = lane; j < f; j += 32) before += a.last[j] >= 0;
      before = __reduce_add_sync(kFull, before);
      const int32_t* row = a.table + (long long)s * a.max_pages;
      int32_t* out = a.table + (long long)d * a.max_pages;
      for (int j = lane; j < full; j += 32) {
        out[j] = row[j];
        atomicAdd(a.shares + row[j], 1);
      }
      if (lane == 0) {
        if (page >= 0) out[full] = to[before];
        a.lens[d] = L;
      }
    }
  }
  copy_pages(p.base[blockIdx.y], p.bytes[blockIdx.y], from, to, total, a.num_pages, a.ws);
}

// ---------------------------------------------------------------------------
// The release of ended sequences
// ---------------------------------------------------------------------------
struct FreeArgs {
  int32_t* table;
  int max_pages;
  int32_t* lens;
  int32_t* shares;
  int num_pages;
  int32_t* stack;
  int32_t* top;
  int capacity;
  const int32_t* seqs;
  int n, B;
  uint32_t* ws;
};

// A warp per sequence: each of its pages loses an owner.  A page without one is left with -1.
__global__ void __launch_bounds__(kThreads) free_rows_kernel(const FreeArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int f = (int)((blockIdx.x * (long long)kThreads + threadIdx.x) >> 5);
  if (f >= a.n) return;  // (whole warps)
  const int s = a.seqs[f];
  bool ok = s >= 0 && s < a.B;
  for (int j = lane; j < f; j += 32)
    if (a.seqs[j] == s) ok = false;  // (named before)
  if (!__all_sync(kFull, ok)) {
    if (lane == 0) atomicOr(a.ws, SV_FLAG_BAD_N);
    return;
  }
  int32_t* row = a.table + (long long)s * a.max_pages;
  bool sound = true;
  for (int j = lane; j < a.max_pages; j += 32) {
    const int id = row[j];
    if (id < 0) continue;
    row[j] = -1;
    if (id >= a.num_pages || atomicSub(a.shares + id, 1) < 0) sound = false;  // (more rows than owners)
  }
  if (lane == 0) a.lens[s] = 0;
  if (!__all_sync(kFull, sound) && lane == 0) atomicOr(a.ws, SV_FLAG_BAD_PAGE);
}

// One CTA: the pages below 0 go on the stack, the lowest id last.
__global__ void __launch_bounds__(kPlanThreads) free_push_kernel(const FreeArgs a) {
  __shared__ int warp_sum[kPlanThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int top = *a.top;
  for (int hi = a.num_pages; hi > 0; hi -= kPlanThreads) {
    const int id = hi - 1 - tid;
    const bool gone = id >= 0 && a.shares[id] < 0;
    const unsigned m = __ballot_sync(kFull, gone);
    if (lane == 0) warp_sum[warp] = __popc(m);
    __syncthreads();
    int v = warp_sum[lane], at = v;  // (32 warps)
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int w = __shfl_up_sync(kFull, at, k);
      if (lane >= k) at += w;
    }
    const int total = __shfl_sync(kFull, at, 31);
    const int place = top + __shfl_sync(kFull, at - v, warp) + __popc(m & ((1u << lane) - 1u));
    if (gone) {
      a.shares[id] = 0;
      if (place >= 0 && place < a.capacity) a.stack[place] = id;
    }
    top += total;
    __syncthreads();
  }
  if (tid == 0) {
    if (top > a.capacity || *a.top < 0) {
      atomicOr(a.ws, SV_FLAG_CAPACITY);
      top = min(top, a.capacity);
    }
    *a.top = top;
  }
}

// ---------------------------------------------------------------------------
// Compaction: with n live pages, those with ids >= n move, in order, to the free
// ids below n.
// ---------------------------------------------------------------------------
struct CompactArgs {
  int num_pages, max_pages, B, prefix_count, words;
  int32_t* table;
  int32_t* prefix;
  int32_t* shares;
  int32_t* stack;
  int32_t* top;
  uint32_t* ws;
  uint32_t* live;   // [words]: a bit per page
  int32_t* before;  // [words]: live pages in front of the word
  int32_t* rank;    // [num_pages], of pages that move
  int32_t* src;     // [num_pages / 2]
  int32_t* dst;
};

__global__ void __launch_bounds__(kThreads) mark_kernel(const CompactArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const long long entries = (long long)a.B * a.max_pages;
  bool sound = true;
  for (long long x = (long long)blockIdx.x * kThreads + threadIdx.x; x < entries + a.prefix_count;
       x += (long long)gridDim.x * kThreads) {
    const int id = x < entries ? a.table[x] : a.prefix[x - entries];
    if (id >= a.num_pages || (x >= entries && id < 0)) sound = false;
    else if (id >= 0) atomicOr(a.live + (id >> 5), 1u << (id & 31));
  }
  if (!sound) atomicOr(a.ws, SV_FLAG_BAD_PAGE);
}

// One CTA: the moves.
__global__ void __launch_bounds__(kPlanThreads) moves_kernel(const CompactArgs a) {
  __shared__ int warp_sum[kPlanThreads / 32];
  __shared__ int below;  // live pages with ids below their number
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int live = 0;
  for (int w0 = 0; w0 < a.words; w0 += kPlanThreads) {
    const int w = w0 + tid;
    const int mine = w < a.words ? __popc(a.live[w]) : 0;
    int up = mine;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int v = __shfl_up_sync(kFull, up, k);
      if (lane >= k) up += v;
    }
    if (lane == 31) warp_sum[warp] = up;
    __syncthreads();
    int v = warp_sum[lane], at = v;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int o = __shfl_up_sync(kFull, at, k);
      if (lane >= k) at += o;
    }
    const int in_front = __shfl_sync(kFull, at - v, warp);  // (of every lane, those without a word too)
    if (w < a.words) a.before[w] = live + in_front + up - mine;
    live += __shfl_sync(kFull, at, 31);
    __syncthreads();
  }
  __syncthreads();
  if (tid == 0)
    below = live == a.num_pages ? live : a.before[live >> 5] + __popc(a.live[live >> 5] & ((1u << (live & 31)) - 1u));
  __syncthreads();
  for (int id = tid; id < a.num_pages; id += kPlanThreads) {
    const uint32_t word = a.live[id >> 5];
    const int in_front = a.before[id >> 5] + __popc(word & ((1u << (id & 31)) - 1u));
    const bool used = word >> (id & 31) & 1;
    if (used && id >= live) {
      a.rank[id] = in_front - below;
      a.src[in_front - below] = id;
    } else if (!used && id < live) {
      a.dst[id - in_front] = id;
    }
  }
  if (tid == 0) {
    a.ws[1] = (uint32_t)(live - below);
    a.ws[2] = (uint32_t)live;
    *a.top = a.num_pages - live;
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ Pools<N> p, const CompactArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int moves = (int)a.ws[1], live = (int)a.ws[2];
  if (blockIdx.y == 0) {
    const long long step = (long long)gridDim.x * kThreads, me = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long entries = (long long)a.B * a.max_pages;
    for (long long x = me; x < entries + a.prefix_count; x += step) {
      int32_t* at = x < entries ? a.table + x : a.prefix + (x - entries);
      const int id = *at;
      if (id >= live && id < a.num_pages) *at = a.dst[a.rank[id]];
    }
    for (long long m = me; m < moves; m += step) {
      const int from = a.src[m];
      a.shares[a.dst[m]] = a.shares[from];
      a.shares[from] = 0;
    }
    for (long long i = me; i < a.num_pages - live; i += step) a.stack[i] = (int32_t)(a.num_pages - 1 - i);
  }
  copy_pages(p.base[blockIdx.y], p.bytes[blockIdx.y], a.src, a.dst, moves, a.num_pages, a.ws);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, void* stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

int done(const char* what, cudaError_t e, std::string* err) {
  if (e == cudaSuccess) return SV_OK;
  *err = std::string(what) + ": " + cudaGetErrorString(e);
  return SV_ERR_CUDA;
}

// CTAs per page array: eight an SM together, and no more than the copies have work for.
dim3 copy_grid(const PagePools& p, long long most_moves) {
  long long largest = 0;
  for (int i = 0; i < p.n; ++i) largest = p.bytes[i] > largest ? p.bytes[i] : largest;
  const long long units = most_moves * ((largest / 16 + 127) / 128);
  long long x = (units + kThreads / 32 - 1) / (kThreads / 32);
  const long long share = (tc::num_sms() * 8LL + p.n - 1) / p.n;
  if (x > share) x = share;
  if (x < 1) x = 1;
  return dim3((unsigned)x, (unsigned)p.n, 1);
}

}  // namespace pages

size_t kv_pages_workspace_bytes(int num_pages, int n) {
  const size_t words = ((size_t)num_pages + 31) / 32;
  const size_t compact = words * 8 + (size_t)num_pages * 8 + 16, fork = (size_t)n * 4;
  return pages::kHead + (compact > fork ? compact : fork);
}

int kv_copy_launch(const PagePools& p, int num_pages, const int32_t* src, const int32_t* dst, int n, void* workspace,
                   void* stream, std::string* err) {
  const dim3 grid = pages::copy_grid(p, n);
  uint32_t* ws = static_cast<uint32_t*>(workspace);
  cudaError_t e;
  if (p.n <= pages::kFew)
    e = pages::launch(pages::copy_kernel<pages::kFew>, grid, pages::kThreads, stream, pages::pools_of<pages::kFew>(p),
                      num_pages, src, dst, n, ws);
  else
    e = pages::launch(pages::copy_kernel<kMaxPools>, grid, pages::kThreads, stream, pages::pools_of<kMaxPools>(p),
                      num_pages, src, dst, n, ws);
  return pages::done("kv_copy_pages launch", e, err);
}

int kv_fork_launch(const PagePools& p, int num_pages, int page_size, int32_t* table, int max_pages, int32_t* lens,
                   int32_t* shares, const int32_t* free_pages, int32_t* free_top, const int32_t* src,
                   const int32_t* dst, int F, int B, void* workspace, void* stream, std::string* err) {
  pages::ForkArgs a;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.F = F;
  a.B = B;
  a.table = table;
  a.lens = lens;
  a.shares = shares;
  a.stack = free_pages;
  a.top = free_top;
  a.src = src;
  a.dst = dst;
  a.ws = static_cast<uint32_t*>(workspace);
  a.last = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + pages::kHead);
  const int per = pages::kThreads / 32;
  cudaError_t e = pages::launch(pages::fork_check_kernel, dim3((F + per - 1) / per), pages::kThreads, stream, a);
  if (e == cudaSuccess) {
    const dim3 grid = pages::copy_grid(p, F);
    if (p.n <= pages::kFew)
      e = pages::launch(pages::fork_apply_kernel<pages::kFew>, grid, pages::kThreads, stream,
                        pages::pools_of<pages::kFew>(p), a);
    else
      e = pages::launch(pages::fork_apply_kernel<kMaxPools>, grid, pages::kThreads, stream,
                        pages::pools_of<kMaxPools>(p), a);
  }
  return pages::done("kv_fork launch", e, err);
}

int kv_free_launch(int32_t* table, int max_pages, int32_t* lens, int32_t* shares, int num_pages, int32_t* free_pages,
                   int32_t* free_top, int free_capacity, const int32_t* seqs, int n, int B, void* workspace,
                   void* stream, std::string* err) {
  pages::FreeArgs a;
  a.table = table;
  a.max_pages = max_pages;
  a.lens = lens;
  a.shares = shares;
  a.num_pages = num_pages;
  a.stack = free_pages;
  a.top = free_top;
  a.capacity = free_capacity;
  a.seqs = seqs;
  a.n = n;
  a.B = B;
  a.ws = static_cast<uint32_t*>(workspace);
  const int per = pages::kThreads / 32;
  cudaError_t e = pages::launch(pages::free_rows_kernel, dim3((n + per - 1) / per), pages::kThreads, stream, a);
  if (e == cudaSuccess) e = pages::launch(pages::free_push_kernel, dim3(1), pages::kPlanThreads, stream, a);
  return pages::done("kv_free launch", e, err);
}

int kv_compact_launch(const PagePools& p, int num_pages, int32_t* table, int max_pages, int B, int32_t* prefix_pages,
                      int prefix_count, int32_t* shares, int32_t* free_pages, int32_t* free_top, void* workspace,
                      void* stream, std::string* err) {
  pages::CompactArgs a;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.B = B;
  a.prefix_count = prefix_count;
  a.words = (num_pages + 31) / 32;
  a.table = table;
  a.prefix = prefix_pages;
  a.shares = shares;
  a.stack = free_pages;
  a.top = free_top;
  a.ws = static_cast<uint32_t*>(workspace);
  a.live = a.ws + pages::kHead / 4;
  a.before = reinterpret_cast<int32_t*>(a.live + a.words);
  a.rank = a.before + a.words;
  a.src = a.rank + num_pages;
  a.dst = a.src + num_pages / 2;
  cudaError_t e = cudaMemsetAsync(a.live, 0, (size_t)a.words * 4, static_cast<cudaStream_t>(stream));
  const long long entries = (long long)B * max_pages + prefix_count;
  long long blocks = (entries + pages::kThreads - 1) / pages::kThreads;
  if (blocks > tc::num_sms() * 8LL) blocks = tc::num_sms() * 8LL;
  if (e == cudaSuccess) e = pages::launch(pages::mark_kernel, dim3((unsigned)blocks), pages::kThreads, stream, a);
  if (e == cudaSuccess) e = pages::launch(pages::moves_kernel, dim3(1), pages::kPlanThreads, stream, a);
  if (e == cudaSuccess) {
    const dim3 grid = pages::copy_grid(p, num_pages / 2 > 0 ? num_pages / 2 : 1);
    if (p.n <= pages::kFew)
      e = pages::launch(pages::compact_kernel<pages::kFew>, grid, pages::kThreads, stream,
                        pages::pools_of<pages::kFew>(p), a);
    else
      e = pages::launch(pages::compact_kernel<kMaxPools>, grid, pages::kThreads, stream, pages::pools_of<kMaxPools>(p),
                        a);
  }
  return pages::done("kv_compact launch", e, err);
}

}  // namespace sv
