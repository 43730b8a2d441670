// The matrix product of few rows with 4-bit weights, group scales, and the
// epilogue of sv_linear:
//
//   z[m][n] = sum_g s[n][g] sum_{k in g} (c[n][k] - zero[n][g]) x[m][k] + bias[n]
//   out[m][n] = act(z[m][n]) + residual[m][n]
//
// Bound by the bytes of W, and next by the integer instructions that take codes apart (half the rate of the
// others).  A code less its zero is an integer of -15 .. 15, exact in fp16: the tensor cores sum a
// group's products in float32 and the scale multiplies that sum, so no weight is rounded.  W is the
// 16-row side of mma.m16n8k16 and x the 8-column side.  A lane's operands of a k step are any four codes
// of a row if x's values follow the same order, so a word of 8 codes (k .. k + 7, as it lies in memory) becomes
// two steps' operands in registers: w & 0x000f000f | 0x64006400 is the pair of fp16 1024 + c and
// w & 0x00f000f0 | 0x64006400 the pair 1024 + 16 c, from which 1024 and the zero are subtracted; 16 goes into
// x.  Five integer instructions for 8 codes (bf16, with 7 bits behind the leading one, takes seven).  x becomes
// fp16 next to a power of two for each of its rows and 128 k: bf16's 8 bits are kept down to 2^-28 of the
// largest of the 128 values, what is smaller is off by at most 2^-36 of it.
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>
#include <string>

#include "sv_act.cuh"
#include "sv_tc.cuh"

namespace sv {
namespace w4 {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 128;  // k of a warp's step
constexpr uint32_t kFull = 0xffffffffu;

struct Args {
  const uint16_t* x;
  long long ldx;
  const uint8_t* W;
  long long ldw;  // bytes
  const uint16_t* scales;
  const uint8_t* zeros;
  const uint16_t* bias;
  const void* res;
  long long ldr;
  void* out;
  long long ldo;
  int act, out_f32, M, N, K, groups;
  unsigned split;  // CTAs that share K
  uint32_t* flags;
  long long clocks;  // of a wait; 0: none is waited for
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t add_f16x2(uint32_t a, uint32_t b) {  // (a difference takes two instructions)
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// w & mask | 1024 in both halves of fp16, in one instruction
template <uint32_t MASK>
__device__ __forceinline__ uint32_t on_1024(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "r"(0x64006400u));
  return r;
}
constexpr uint32_t kLess1024 = 0xe400e400u;  // -1024 twice; a zero in its low bits makes it -(1024 + zero)

// Two pairs of codes of a word less their zeros: c of the lowest four bits of each half, 16 c of the next four.
__device__ __forceinline__ uint32_t low_codes(uint32_t w, uint32_t less) { return add_f16x2(on_1024<0x000f000fu>(w), less); }
__device__ __forceinline__ uint32_t high_codes(uint32_t w, uint32_t less) { return add_f16x2(on_1024<0x00f000f0u>(w), less); }

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A tile's outputs from the sums part[column][row] of a cluster's CTAs, added in the order of their ranks; each
// CTA writes a share of them.
template <int ROWS, int THREADS>
__device__ __forceinline__ void finish(const Args& a, const float* part, int n0, int m0, int cols, unsigned rank) {
  for (int x = (int)rank * THREADS + (int)threadIdx.x; x < ROWS * cols; x += (int)a.split * THREADS) {
    const int n = n0 + x % ROWS;
    const long long m = m0 + x / ROWS;
    float z[1] = {0.f};
    if (a.split > 1) {
      for (unsigned q = 0; q < a.split; ++q) z[0] += tc::ld_cluster(tc::cluster_addr(part + x, q));
    } else {
      z[0] = part[x];
    }
    if (n >= a.N) continue;
    if (a.bias) z[0] += __uint_as_float((uint32_t)a.bias[n] << 16);
    lin::activate(z, a.act);
    if (a.out_f32) {
      if (a.res) z[0] += static_cast<const float*>(a.res)[m * a.ldr + n];
      static_cast<float*>(a.out)[m * a.ldo + n] = z[0];
    } else {
      if (a.res) z[0] += __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.res)[m * a.ldr + n] << 16);
      static_cast<uint16_t*>(a.out)[m * a.ldo + n] = __bfloat16_as_ushort(__float2bfloat16_rn(z[0]));
    }
  }
}

__device__ __forceinline__ void cp16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t to, const void* from, bool there) {  // zeros if it is not
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}

// A warp's step: 16 rows of W by 128 k, 64 bytes a row, in rows of 80 bytes (a lane's words of its rows g and
// g + 8, VEC words at a time, then meet 32 banks).
constexpr int kPitch = 80;
constexpr int kStages = 8;   // of a warp
constexpr int kAhead = 6;    // steps on their way
constexpr int kStageBytes = 16 * kPitch;

// 1 x 16384 x 4096 in groups of 128: 14.0 us a call in a row of calls whose W come from HBM, where its 34 MB take 5
// (alone, behind an emptied L2, 19 to 21 us with the launch); the start, the ends of the chunks' chains and the
// instructions (46% of the issue slots) share the rest.
constexpr int kTiles = 4;    // of a CTA: more share the work on x, fewer want fewer registers
constexpr int kRows = 16 * kTiles;
constexpr int kCtas = 2;     // of an SM

// Up to 8 rows of x.  VEC words (VEC * 32 k) are a group.
template <int VEC>
__global__ void __launch_bounds__(kThreads, kCtas) rows_kernel(const __grid_constant__ Args a) {
  constexpr int COLS = 8, L = 4 / VEC;
  extern __shared__ __align__(16) uint8_t ring[];  // [kWarps][kStages][kStageBytes]
  __shared__ float part[COLS][kRows];
  float (*red)[COLS][kRows] = reinterpret_cast<float (*)[COLS][kRows]>(ring);  // behind the products
  static_assert(kWarps * kStages * kStageBytes >= kWarps * COLS * kRows * 4, "the warps' sums fit over the ring");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  pdl_launch_dependents();
  pdl_wait();
  const unsigned slab = blockIdx.x / a.split, rank = blockIdx.x - slab * a.split;
  const int n0 = (int)slab * kRows;
  const int chunks = (a.K + kChunk - 1) / kChunk, workers = (int)a.split * kWarps, me = (int)rank * kWarps + warp;
  // (neighbours in a row of W are read at about the same time: runs of 64 bytes alone are slow)
  const int c0 = me, c1 = chunks;
  const uint32_t base = smem_addr(ring) + warp * kStages * kStageBytes;
  // bytes 16 t .. of rows g and g + 8 of a tile
  const int n_mine = n0 + g;
  const bool full = n0 + kRows <= a.N;  // (behind the last row the last one's codes again)
  const long long by8 = 8 * a.ldw;
  const uint8_t* next = a.W + n_mine * a.ldw + t * 16 + (long long)c0 * (kChunk / 2);  // of the next step
  const uint32_t to = base + g * kPitch + t * 16;
  // tile i of chunk c, in turn: slot `at` of the ring
  auto issue = [&](int c, int i, int at) {
    if (c < c1) {
      const uint32_t where = to + at * kStageBytes;
      if (full && (VEC == 4 || (c + 1) * kChunk <= a.K)) {
        cp16(where, next);
        cp16(where + 8 * kPitch, next + by8);
      } else {
        const bool there = c * kChunk + t * 32 < a.K;
        const uint8_t* p = a.W + (there ? (long long)c * (kChunk / 2) + t * 16 : 0);
        cp16(where, p + min(n_mine + 16 * i, a.N - 1) * a.ldw, there);
        cp16(where + 8 * kPitch, p + min(n_mine + 16 * i + 8, a.N - 1) * a.ldw, there);
      }
      next += i == kTiles - 1 ? workers * (kChunk / 2) - (2 * kTiles - 2) * by8 : 2 * by8;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // What a chunk takes beside its codes is read a chunk ahead, all of it before any is used (a condition around a
  // load makes it wait for the one before): behind the last chunk that chunk's again, behind the last row of x that
  // row.  Of the kTiles * L (scale, zero) of row g, and of row g + 8, of the chunk, lane t reads the q-th with
  // q % 4 = t; at their use they come by shuffle.
  constexpr int Q = kTiles * L / 4;
  auto load_scales = [&](int c, uint16_t (&scale)[Q][2], uint8_t (&zero)[Q][2]) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int one = q * 4 + t;
        const uint32_t at = (uint32_t)min(n_mine + 16 * (one / L) + 8 * r, a.N - 1) * a.groups +
                            (uint32_t)min(c * L + one % L, a.groups - 1);
        scale[q][r] = __ldg(a.scales + at);
        zero[q][r] = __ldg(a.zeros ? a.zeros + at : reinterpret_cast<const uint8_t*>(a.scales + at));
      }
  };
  const uint16_t* xrow = a.x + min(g, a.M - 1) * a.ldx;
  auto load_x = [&](int c, uint4 (&v)[4]) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int k = c * kChunk + w / VEC * 32 * VEC + t * 8 * VEC + w % VEC * 8;
      v[w] = __ldg(reinterpret_cast<const uint4*>(xrow + (VEC == 4 ? k : min(k, a.K - 8))));
    }
  };

  float total[kTiles][4] = {};
  uint4 xn[4];
  uint16_t sn[Q][2];
  uint8_t zn[Q][2];
#pragma unroll
  for (int st = 0; st < kAhead; ++st) issue(c0 + st / kTiles * workers, st % kTiles, st);
  load_x(min(c0, chunks - 1), xn);
  load_scales(min(c0, chunks - 1), sn, zn);
  int slot = 0;  // of the chunk's first step
#pragma unroll 1
  for (int c = c0; c < c1; c += workers) {
    uint32_t b[4][4], sz[Q][2];  // (a scale in the high half, its zero in the low byte)
    float undo[2];  // x's power of two, of the lane's columns
    {
      uint32_t top = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (VEC < 4 && c * kChunk + w / VEC * 32 * VEC + t * 8 * VEC >= a.K) xn[w] = make_uint4(0, 0, 0, 0);
        const uint4 v = xn[w];
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                     __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
      }
      top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 2));
      const int ex = (int)(max(top & 0xffffu, top >> 16) >> 7);  // biased exponent of the largest value
      // the largest value becomes 2^15 or more, below 2^16, with a factor of at most 2^126 (which makes every bf16
      // value a multiple of 2^-7); the high codes' sixteenth of it loses four bits at the lower end.  (Exponents
      // subtracted in integers were no faster, 14.2 us for 14.0, and had no subnormal values.)
      const int fb = min(269 - ex, 253);
      const float up = __uint_as_float((uint32_t)fb << 23), up16 = up * 0.0625f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint4 v = xn[w];
        b[w][0] = half2_of(bf16_lo(v.x) * up, bf16_lo(v.z) * up);
        b[w][1] = half2_of(bf16_hi(v.x) * up16, bf16_hi(v.z) * up16);
        b[w][2] = half2_of(bf16_lo(v.y) * up, bf16_lo(v.w) * up);
        b[w][3] = half2_of(bf16_hi(v.y) * up16, bf16_hi(v.w) * up16);
      }
      // NaN for a row that is not finite
      const float f = ex == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(254 - fb) << 23);
#pragma unroll
      for (int j = 0; j < 2; ++j) undo[j] = __shfl_sync(kFull, f, (2 * t + j) * 4);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int r = 0; r < 2; ++r) sz[q][r] = (uint32_t)sn[q][r] << 16 | (a.zeros ? zn[q][r] : 8u);
    load_x(min(c + workers, c1 - 1), xn);
    load_scales(min(c + workers, c1 - 1), sn, zn);
    const uint32_t here = base + g * kPitch + t * VEC * 4;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      issue(c + (i + kAhead) / kTiles * workers, (i + kAhead) % kTiles, (slot + i + kAhead) & (kStages - 1));
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
      __syncwarp();
      uint32_t u[4], v[4];
#pragma unroll
      for (int l = 0; l < L; ++l) {
        const uint32_t p = here + ((slot + i) & (kStages - 1)) * kStageBytes + l * VEC * 16;
        if constexpr (VEC == 4) {
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                       : "r"(p)
                       : "memory");
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                       : "r"(p + 8 * kPitch)
                       : "memory");
        } else if constexpr (VEC == 2) {
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(u[2 * l]), "=r"(u[2 * l + 1]) : "r"(p) : "memory");
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[2 * l]), "=r"(v[2 * l + 1]) : "r"(p + 8 * kPitch) : "memory");
        } else {
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(u[l]) : "r"(p) : "memory");
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[l]) : "r"(p + 8 * kPitch) : "memory");
        }
      }
#pragma unroll
      for (int l = 0; l < L; ++l) {
        const uint32_t sz0 = __shfl_sync(kFull, sz[(i * L + l) / 4][0], (lane & ~3) + (i * L + l) % 4);
        const uint32_t sz1 = __shfl_sync(kFull, sz[(i * L + l) / 4][1], (lane & ~3) + (i * L + l) % 4);
        const uint32_t z0 = (sz0 & 255u) * 0x10001u + kLess1024, z1 = (sz1 & 255u) * 0x10001u + kLess1024;
        const uint32_t y0 = (sz0 & 255u) * 0x100010u + kLess1024, y1 = (sz1 & 255u) * 0x100010u + kLess1024;
        float acc[4] = {}, acc2[4] = {};  // (two chains of products)
#pragma unroll
        for (int w = l * VEC; w < (l + 1) * VEC; ++w) {
          mma_f16(acc, low_codes(u[w], z0), low_codes(v[w], z1), high_codes(u[w], y0), high_codes(v[w], y1), b[w][0], b[w][1]);
          const uint32_t u8 = u[w] >> 8, v8 = v[w] >> 8;
          mma_f16(acc2, low_codes(u8, z0), low_codes(v8, z1), high_codes(u8, y0), high_codes(v8, y1), b[w][2], b[w][3]);
        }
        const float s0 = bf16_hi(sz0), s1 = bf16_hi(sz1);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          total[i][e] = __fmaf_rn(e < 2 ? s0 : s1, (acc[e] + acc2[e]) * undo[e & 1], total[i][e]);
      }
      __syncwarp();
    }
    slot = (slot + kTiles) & (kStages - 1);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // (the ring is read no more)
  const int cols = a.M;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (2 * t + j < cols) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        red[warp][2 * t + j][i * 16 + g] = total[i][j];
        red[warp][2 * t + j][i * 16 + g + 8] = total[i][2 + j];
      }
    }
  __syncthreads();
  for (int x = tid; x < kRows * cols; x += kThreads) {
    float z = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) z += red[w][x / kRows][x % kRows];
    part[x / kRows][x % kRows] = z;
  }
  if (a.split > 1) tc::cluster_sync();
  else __syncthreads();
  finish<kRows, kThreads>(a, part[0], n0, 0, cols, rank);
  if (a.split > 1) tc::cluster_sync();  // (no CTA leaves while its sums are read)
}

// ---------------------------------------------------------------------------
// More rows of x: the 5th-generation tensor cores.  A CTA takes 128 rows of W by TM rows of x and a part of K, in
// blocks of 128 k.  Codes and x arrive by TMA; four warps of a block make its codes bf16 integers (code less zero,
// exact) in tensor memory, where the 128-row operand may stand (through shared memory its bytes were the bound); a thread issues
// the groups' products, each group's into an accumulator of tensor memory of its own; four or eight warps take those
// out, times the groups' scales, and add them to their float32 sums in registers.  64 x 16384 x 4096 in groups of 128:
// 20.8 us, 16 x 8192 x 8192 in groups of 64: 19.7 us a call in a row of calls whose W come from HBM, where its 34 MB
// take 5 (alone, behind an emptied L2, 29 and 27 us with the launch); bound by the way of a block through these warps (its parts take 400 to 800 cycles each, and four are under way), next by the instructions that take codes
// apart.  mma.sync took 66 us for the first, since each warp then multiplies all rows of x and the codes have to be
// taken apart again for every 8 of them.
// ---------------------------------------------------------------------------
constexpr int kTeams = 4;            // a team takes every fourth block, of the two issuing warps each every other one
constexpr int kCodeWarps = 4;        // of a team: a row of W a thread
constexpr int kLoadWarp = 16, kMmaWarp = 17, kSumWarp = 19;
constexpr int kTcRows = 128;
constexpr int kRaw = 8;              // blocks of codes and x on their way
constexpr int kRawBytes = kTcRows * 64;
constexpr int kSides = 4;            // blocks of bf16 codes ready for their products, or in them

template <int TM, int GROUP>
struct TcShape {
  static constexpr int kPer = 128 / GROUP;  // groups of a block
  // Groups that are told to be done at once: those of a block, as long as two such units fit.  (A commit keeps the
  // issuing warp for some 200 cycles, and a wait costs as much.)
  static constexpr int kUnit = kPer * TM <= 128 ? kPer : 128 / TM;
  static constexpr int kAccs = kUnit * TM <= 32 ? 8 : 256 / (kUnit * TM);  // units of accumulators
  // A wait tells a phase from the one before only if the waiter has seen that one end.  So a ring's slot is always
  // waited for by the same warp: two warps issue, taking turns, only where the accumulators hold two blocks.
  static constexpr int kIssuers = kAccs * kUnit >= 2 * kPer ? 2 : 1;
  static_assert(kSides % kTeams == 0 && kRaw % kTeams == 0 && kAccs * kUnit % (kIssuers * kPer) == 0, "waits in turn");
  static constexpr int kX = 2 * TM * 128;  // of a block
  static constexpr int kPart = TM * kTcRows * 4;
  static constexpr int kStage = kX + kRawBytes;
  static constexpr int kTiles = kRaw * kStage, kSmem = (kTiles > kPart ? kTiles : kPart) + 1024;
  static constexpr uint32_t kCodes = 256;  // columns of the accumulators; then 64 of codes for each side
  static constexpr uint32_t kColumns = 512;
  static_assert(kAccs * kUnit * TM <= (int)kCodes && kCodes + kSides * 64 <= kColumns, "tensor memory");
  static constexpr int kSumWarps = TM == 64 ? 8 : 4, kColumnsEach = TM * 4 / kSumWarps;
  static constexpr int kThreads = (kSumWarp + kSumWarps) * 32;
};

// Pair J of a word's four pairs of bf16 (code less zero); w4 = w >> 4, less = -(128 + zero) twice.
template <int J>
__device__ __forceinline__ uint32_t pair_of(uint32_t w, uint32_t w4, uint32_t less) {
  uint32_t r = __byte_perm(w, w4, 0x0400 + J * 0x0101);  // byte J of both, one in each half
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(r), "n"(0x000f000f), "r"(0x43004300u));
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(less));
  return r;
}
// true in one lane of a whole warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
// eight columns of the warp's 32 lanes into tensor memory
__device__ __forceinline__ void st8(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f,
                                    uint32_t g, uint32_t h) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(a), "r"(b),
               "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h)
               : "memory");
}

template <int TM, int GROUP>
__global__ void __launch_bounds__(TcShape<TM, GROUP>::kThreads, 1) tile_kernel(
    const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const __grid_constant__ Args a) {
  using S = TcShape<TM, GROUP>;
  constexpr int PER = S::kPer, UNIT = S::kUnit;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t raw_full[kRaw], raw_empty[kRaw], a_full[kSides], a_empty[kSides];
  __shared__ __align__(8) uint64_t acc_full[S::kAccs], acc_empty[S::kAccs], done;
  __shared__ uint32_t tmem_base;
  __shared__ int failed, issued;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);  // (the same in the whole warp, and known to be)
  const unsigned block = blockIdx.x / a.split, rank = blockIdx.x - block * a.split;
  const int blocks = (a.M + TM - 1) / TM, slab = (int)(block / blocks);
  const int n0 = slab * kTcRows, m0 = (int)(block - slab * blocks) * TM;
  const int all = (a.K + 127) / 128;
  const int b0 = (int)((long long)all * rank / a.split), b1 = (int)((long long)all * (rank + 1) / a.split);
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t at_x = smem_addr(tiles), at_raw = at_x + S::kX;  // of the first stage
  if (tid == 0) {
    for (int s = 0; s < kRaw; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 1);
    }
    for (int s = 0; s < kSides; ++s) {
      mbar_init(&a_full[s], kCodeWarps);
      mbar_init(&a_empty[s], 1);
    }
    for (int s = 0; s < S::kAccs; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], S::kSumWarps);
    }
    mbar_init(&done, 2);
    failed = issued = 0;
    fence_mbar_init();
    tc::prefetch_map(&tmW);
    tc::prefetch_map(&tmX);
  }
  if (warp == kLoadWarp) tc::alloc<1>(&tmem_base, S::kColumns);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_base;
  pdl_launch_dependents();  // (behind the allocation: a dependent cannot take this CTA's columns)
  pdl_wait();
  // a wait of at most about a second, none at all if `clocks` is 0; who gives up leaves its loop
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (a.clocks > 0 && tc::wait_bounded(bar, parity, a.clocks)) return true;
    failed = 1;
    return false;
  };
  float total[S::kColumnsEach] = {};

  if (warp < kLoadWarp) {
    const int team = warp / kCodeWarps, r = tid - team * kCodeWarps * 32, n = min(n0 + r, a.N - 1);
    // (without zeros the bytes of W are loaded in their place and not used: a choice at the load would wait for it)
    const bool has_zeros = a.zeros != nullptr;
    const uint8_t* zrow = has_zeros ? a.zeros + (uint32_t)n * a.groups : a.W + n * a.ldw;
    auto load_zeros = [&](int b, uint32_t (&z)[PER]) {
#pragma unroll
      for (int q = 0; q < PER; ++q) z[q] = __ldg(zrow + min(b * PER + q, a.groups - 1));
    };
    uint32_t zn[PER];
    load_zeros(b0 + team, zn);
    const uint32_t to = tmem + ((uint32_t)((warp & 3) * 32) << 16) + S::kCodes;  // (r's lane)
    const uint32_t raw_row = r * 64, raw_flip = (uint32_t)(r >> 1) & 3;
    for (int b = b0 + team, g = team; b < b1; b += kTeams, g += kTeams) {
      const int s = g % kRaw, side = g % kSides;
      uint32_t less[PER];
#pragma unroll
      for (int q = 0; q < PER; ++q) less[q] = (has_zeros ? zn[q] : 8u) * 0x10001u + 0xc300c300u;
      load_zeros(b + kTeams, zn);
      if (g >= kSides && !__all_sync(kFull, wait(&a_empty[side], (g / kSides - 1) & 1))) break;  // (the whole warp)
      tc::fence_after();
      if (!__all_sync(kFull, wait(&raw_full[s], g / kRaw & 1))) break;
#pragma unroll
      for (int h = 0; h < 4; ++h) {  // 32 k
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(at_raw + s * S::kStage + raw_row + (((uint32_t)h ^ raw_flip) << 4))
                     : "memory");
        const uint32_t l = less[h * PER / 4];
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          const uint32_t u = w[c], v = w[c + 1], u4 = u >> 4, v4 = v >> 4;
          st8(to + side * 64 + h * 16 + c * 4, pair_of<0>(u, u4, l), pair_of<1>(u, u4, l), pair_of<2>(u, u4, l),
              pair_of<3>(u, u4, l), pair_of<0>(v, v4, l), pair_of<1>(v, v4, l), pair_of<2>(v, v4, l), pair_of<3>(v, v4, l));
        }
      }
      tc::st_wait();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&a_full[side]);
    }
  } else if (warp == kLoadWarp) {
    if (lane == 0) {
      int g = 0;
      for (int b = b0; b < b1; ++b, ++g) {
        const int s = g % kRaw;
        if (g >= kRaw && !wait(&raw_empty[s], (g / kRaw - 1) & 1)) break;
        mbar_arrive_expect_tx(&raw_full[s], S::kStage);
        tc::tma_load(tiles + s * S::kStage + S::kX, &tmW, b * 64, n0, &raw_full[s]);
        tc::tma_load(tiles + s * S::kStage, &tmX, b * 128, m0, &raw_full[s]);
        tc::tma_load(tiles + s * S::kStage + S::kX / 2, &tmX, b * 128 + 64, m0, &raw_full[s]);
      }
      issued = g;
    }
  } else if (warp < kSumWarp) {
    // The whole warp takes this way, so that descriptors are computed in uniform registers, where the instruction
    // wants them; one lane issues.
    constexpr uint32_t id = tc::idesc(false, false, 128, TM);
    const bool elected = elect_one();
    const int team = warp - kMmaWarp;
    bool ok = true;
    for (int b = b0 + team, g = team; b < b1 && ok && team < S::kIssuers; b += S::kIssuers, g += S::kIssuers) {
      const int side = g % kSides, s = g % kRaw;
      const uint32_t block_a = tmem + S::kCodes + side * 64, block_x = tc::desc_low(at_x, 16) + s * (S::kStage >> 4);
      ok = __all_sync(kFull, wait(&raw_full[s], g / kRaw & 1) && wait(&a_full[side], g / kSides & 1));
      tc::fence_after();
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        if (!ok || b * PER + q >= a.groups) break;
        const int acc = (g * PER + q) / UNIT, slot = acc % S::kAccs;
        if (q % UNIT == 0) {
          ok = acc < S::kAccs || __all_sync(kFull, wait(&acc_empty[slot], (acc / S::kAccs - 1) & 1));
          if (!ok) break;
          tc::fence_after();
        }
        const uint32_t d = tmem + (slot * UNIT + q % UNIT) * TM;
        if (elected) {
#pragma unroll
          for (int i = 0; i < GROUP / 16; ++i) {
            constexpr int kSteps = GROUP / 16;
            const int k = q * kSteps + i;  // of the block's eight steps
            tc::mma_ts_low(d, block_a + k * 8, block_x + (((k >> 2) * TM * 128 + (k & 3) * 32) >> 4), id, i != 0);
          }
          if (q % UNIT == UNIT - 1 || b * PER + q + 1 == a.groups) tc::commit<1>(smem_addr(&acc_full[slot]));
        }
      }
    }
    if (elected) tc::commit<1>(smem_addr(&done));  // (nothing arrives behind the CTA's end)
    if (!tc::wait_bounded(&done, 0)) failed = 1;
  } else {
    const int quad = warp & 3, n = min(n0 + quad * 32 + lane, a.N - 1);
    const uint16_t* srow = a.scales + (uint32_t)n * a.groups;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + (warp - kSumWarp) / 4 * S::kColumnsEach;
    const int g0 = b0 * PER, g1 = min(b1 * PER, a.groups);
    uint32_t next[UNIT];
#pragma unroll
    for (int i = 0; i < UNIT; ++i) next[i] = __ldg(srow + min(g0 + i, a.groups - 1));
    for (int group = g0, acc = 0; group < g1; group += UNIT, ++acc) {
      float s[UNIT];
#pragma unroll
      for (int i = 0; i < UNIT; ++i) {
        s[i] = __uint_as_float(next[i] << 16);
        next[i] = __ldg(srow + min(group + UNIT + i, a.groups - 1));
      }
      const int slot = acc % S::kAccs;
      if (!__all_sync(kFull, wait(&acc_full[slot], acc / S::kAccs & 1))) break;
      tc::fence_after();
      if (tid == kSumWarp * 32 && ((group + UNIT) % PER == 0 || group + UNIT >= g1)) {
        // the block's products are done, and with them its codes and x
        const int g = group / PER - b0;
        tc::fence_before();
        mbar_arrive(&a_empty[g % kSides]);
        mbar_arrive(&raw_empty[g % kRaw]);
      }
      constexpr int kPieces = S::kColumnsEach / 16, kAll = UNIT * kPieces, kTwo = kAll > 1 ? 2 : 1;
#pragma unroll
      for (int p = 0; p < kAll; p += kTwo) {
        uint32_t v[kTwo][16];
#pragma unroll
        for (int j = 0; j < kTwo; ++j)
          tc::ld16(lanes + (slot * UNIT + (p + j) / kPieces) * TM + (p + j) % kPieces * 16, v[j]);
#pragma unroll
        for (int j = 0; j < kTwo; ++j) {
          tc::ld_wait(v[j]);
          const int i = (p + j) / kPieces, c = (p + j) % kPieces * 16;
          if (group + i < g1) {  // (behind the last group nothing was written)
#pragma unroll
            for (int e = 0; e < 16; ++e) total[c + e] = __fmaf_rn(s[i], __uint_as_float(v[j][e]), total[c + e]);
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[slot]);
    }
  }
  __syncthreads();
  const bool lost = failed != 0;  // (the same in every thread)
  if (lost) {  // a wait ran out: copies and products on their way end first, and the tile is NaN
    if (tid == 0) {
      atomicOr(a.flags, SV_FLAG_TIMEOUT);
      for (int g = issued > kRaw ? issued - kRaw : 0; g < issued; ++g) tc::wait_bounded(&raw_full[g % kRaw], g / kRaw & 1);
      tc::wait_bounded(&done, 0);
    }
    __syncthreads();
  }
  float* part = reinterpret_cast<float*>(tiles);  // [TM][128], over the rings
  if (warp >= kSumWarp) {
#pragma unroll
    for (int c = 0; c < S::kColumnsEach; ++c)
      part[((warp - kSumWarp) / 4 * S::kColumnsEach + c) * kTcRows + (warp & 3) * 32 + lane] =
          lost ? __uint_as_float(0x7fffffffu) : total[c];
  }
  if (a.split > 1) tc::cluster_sync();
  else __syncthreads();
  finish<kTcRows, S::kThreads>(a, part, n0, m0, min(TM, a.M - m0), rank);
  if (a.split > 1) tc::cluster_sync();  // (no CTA leaves while its sums are read)
  tc::fence_before();
  __syncthreads();
  if (warp == kLoadWarp) tc::dealloc<1>(tmem, S::kColumns);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Slabs of W times parts of K (at most 8, a cluster): as many CTAs as the card holds at once, as long as each of
// `workers` of a CTA keeps a step of 128 k.
template <typename Kernel, typename... A>
cudaError_t launch(Kernel* kernel, std::atomic<int>* ready, long long slabs, int per_sm, int workers, int threads, int smem,
                   Args a, void* stream, const A&... map) {
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready[dev].store(1, std::memory_order_release);
  }
  const long long fit = (long long)tc::num_sms() * per_sm / slabs;
  const int steps = (a.K + 127) / 128;
  a.split = (unsigned)(fit < 1 ? 1 : fit > 8 ? 8 : fit);
  while (a.split > 1 && steps < (int)a.split * workers) --a.split;
  if (slabs * a.split > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(slabs * a.split), 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, map..., a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int VEC>
cudaError_t launch_rows(const Args& a, void* stream) {
  static std::atomic<int> ready[kMaxDevices];
  const long long slabs = (a.N + kRows - 1LL) / kRows;
  return launch(rows_kernel<VEC>, ready, slabs, kCtas, kWarps, kThreads, kWarps * kStages * kStageBytes, a, stream);
}

template <int TM, int GROUP>
cudaError_t launch_tiles(const Args& a, const CUtensorMap& codes, const CUtensorMap& x, void* stream) {
  static std::atomic<int> ready[kMaxDevices];
  const long long slabs = ((a.N + kTcRows - 1LL) / kTcRows) * ((a.M + TM - 1LL) / TM);
  using S = TcShape<TM, GROUP>;
  return launch(tile_kernel<TM, GROUP>, ready, slabs, 1, 2, S::kThreads, S::kSmem, a, stream, codes, x);
}

bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* at, long long cols, long long rows, long long pitch,
            int box_cols, int box_rows, CUtensorMapSwizzle swizzle, std::string* err) {
  const tc::EncodeTiledFn enc = tc::encoder(err);
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)pitch};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, estr[2] = {1, 1};
  const CUresult r = enc(map, type, 2, const_cast<void*>(at), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) *err = "linear_w4: cuTensorMapEncodeTiled failed with CUresult " + std::to_string((int)r);
  return r == CUDA_SUCCESS;
}

// Rows of K / 2 bytes of codes in boxes of 64 bytes by 128 rows, of K values of x in boxes of 64 by TM; zeros outside.
template <int TM>
cudaError_t tiles_by_group(const Args& a, int group, void* stream, std::string* err) {
  CUtensorMap codes, x;
  if (!encode(&codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.W, a.K / 2, a.N, a.ldw, 64, kTcRows, CU_TENSOR_MAP_SWIZZLE_64B, err) ||
      !encode(&x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.K, a.M, a.ldx * 2, 64, TM, CU_TENSOR_MAP_SWIZZLE_128B, err))
    return cudaErrorInvalidValue;
  return group == 128  ? launch_tiles<TM, 128>(a, codes, x, stream)
         : group == 64 ? launch_tiles<TM, 64>(a, codes, x, stream)
                       : launch_tiles<TM, 32>(a, codes, x, stream);
}

}  // namespace w4

size_t linear_w4_workspace_bytes(int, int, int) { return 256; }

int linear_w4_launch(const LinearW4Launch& L, std::string* err) {
  w4::Args a;
  a.x = static_cast<const uint16_t*>(L.x);
  a.ldx = L.ldx;
  a.W = static_cast<const uint8_t*>(L.W);
  a.ldw = L.ldw;
  a.scales = static_cast<const uint16_t*>(L.scales);
  a.zeros = static_cast<const uint8_t*>(L.zeros);
  a.bias = static_cast<const uint16_t*>(L.bias);
  a.res = L.residual;
  a.ldr = L.ldr;
  a.out = L.out;
  a.ldo = L.ldo;
  a.act = L.act;
  a.out_f32 = L.out_dtype == SV_F32;
  a.M = L.M;
  a.N = L.N;
  a.K = L.K;
  a.groups = L.K / L.group;
  a.flags = static_cast<uint32_t*>(L.workspace);
  a.clocks = L.wait_tries > 0 ? tc::kWaitClocks : 0;
  cudaError_t e;
  if (L.M <= 8) {
    e = L.group == 128  ? w4::launch_rows<4>(a, L.stream)
        : L.group == 64 ? w4::launch_rows<2>(a, L.stream)
                        : w4::launch_rows<1>(a, L.stream);
  } else {
    e = L.M <= 16   ? w4::tiles_by_group<16>(a, L.group, L.stream, err)
        : L.M <= 32 ? w4::tiles_by_group<32>(a, L.group, L.stream, err)
                    : w4::tiles_by_group<64>(a, L.group, L.stream, err);
  }
  if (e != cudaSuccess && !err->empty()) return SV_ERR_CUDA;
  if (e == cudaSuccess) return SV_OK;
  *err = std::string("linear_w4 launch: ") + cudaGetErrorString(e);
  return SV_ERR_CUDA;
}

}  // namespace sv
