// How the key tiles of the 4-bit attention are shared out among its warps, and which
// of them join a group's parts: arithmetic of the kernel that the host can run too.
//
// The groups (sequence, key head, block of query rows) lie in a row, each as long as its
// tiles and kGroupCost; warp w has the units [w share, (w + 1) share) of it.  A group whose
// tiles lie in one share is whole, another is cut into a part for each of its warps w0 .. w1.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SV_HOST_DEVICE inline
#endif

namespace sv {
namespace kv4 {

// What a group costs beside its tiles, in tiles: Q, the stores, the way to the next.  The 256 sequences take 135.5 /
// 128.9 / 126.8 / 129.1 us in a graph with 3 / 5 / 9 / 13.
constexpr int kGroupCost = 9;
constexpr int kMinShare = 7;       // of a warp (5: 4 sequences of a round 21.2 us, 7: 19.7)
constexpr int kJoin = 16;          // parts that are joined at once

// a / b, in 32 bits where they fit (a third of the time).
SV_HOST_DEVICE unsigned long long quotient(unsigned long long a, unsigned long long b) {
  return (a | b) >> 32 ? a / b : (uint32_t)a / (uint32_t)b;
}

SV_HOST_DEVICE unsigned long long share_of(unsigned long long total, unsigned warps) {
  const unsigned long long share = quotient(total + warps - 1, warps);
  return share < kMinShare ? kMinShare : share;
}

// Where a warp's part of a group lies: the first place of a group that began in front of the warp's
// share, the second of one that begins inside it.
SV_HOST_DEVICE int part_place(unsigned warp, unsigned long long share, unsigned long long group) {
  return warp * share >= group ? 0 : 1;
}

// The run of up to kJoin neighbouring warps of a cut group whose parts are joined together: `worker`'s.
struct Run {
  unsigned w0;     // the group's first warp
  unsigned first;  // the run's first warp, which its finished parts are counted at
  int n;           // warps of the run; the only one of a run of one counts nothing
  unsigned runs;   // of the group; their joins are counted at w0
};
// Each word then belongs to one group.  Of the cut groups one at most begins in a warp's share, so a group's
// first run and the joins of its runs are alone at w0, and one at most goes on from the share before, so a later
// run is alone among these at `first`.  A first run and a later one meet only where the one group's w0 is the
// other's last warp, and there the later run is that warp by itself.
SV_HOST_DEVICE Run run_of(unsigned long long group, int tiles, unsigned long long share, unsigned worker) {
  Run r;
  r.w0 = (unsigned)quotient(group + kGroupCost, share);
  const unsigned w1 = (unsigned)quotient(group + kGroupCost + tiles - 1, share);
  r.first = r.w0 + (worker - r.w0) / kJoin * kJoin;
  r.n = w1 - r.first + 1 < kJoin ? (int)(w1 - r.first + 1) : kJoin;
  r.runs = (w1 - r.w0) / kJoin + 1;
  return r;
}

}  // namespace kv4
}  // namespace sv
