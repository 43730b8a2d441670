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
// fp16 next to a power of two for each of its rows and 128 k: bf16's 8 bits are kept down to 2^-25 of the
// largest of the 128 values, what is smaller counts as 0.
#include <atomic>
#include <cstdint>

#include "sv_act.cuh"
#include "sv_tc.cuh"

namespace sv {
namespace w4 {

constexpr int kWarps = 4;
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

// A pair of bf16 whose exponents lie in `low` (both halves, bf16 with no bits behind the leading one) .. low + 30
// as fp16 with exponents 0 .. 30; smaller values become 0.
__device__ __forceinline__ uint32_t to_f16x2(uint32_t v, uint32_t low) {
  return (__vmaxu2(v & 0x7fff7fffu, low) - low) << 3 | (v & 0x80008000u);
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

// NT blocks of 8 rows of x, tiles of 16 rows of W (as many as registers hold the sums of); VEC words (VEC * 32 k)
// are a group.
template <int NT>
struct Shape {
  static constexpr int kTiles = NT == 1 ? 8 : 4, kRows = 16 * kTiles;
  static constexpr int kCtas = 3;  // of an SM
};

template <int NT, int VEC>
__global__ void __launch_bounds__(kThreads, Shape<NT>::kCtas) rows_kernel(const __grid_constant__ Args a) {
  constexpr int COLS = 8 * NT, L = 4 / VEC, kTiles = Shape<NT>::kTiles, kRows = Shape<NT>::kRows;
  __shared__ __align__(16) uint8_t ring[kWarps][kStages][kStageBytes];
  __shared__ float part[COLS][kRows];
  float (*red)[COLS][kRows] = reinterpret_cast<float (*)[COLS][kRows]>(ring);  // behind the products
  static_assert(sizeof(ring) >= kWarps * COLS * kRows * 4, "the warps' sums fit over the ring");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  pdl_wait();
  const unsigned block = blockIdx.x / a.split, rank = blockIdx.x - block * a.split;
  const int blocks = (a.M + COLS - 1) / COLS, slab = (int)(block / blocks);
  const int n0 = slab * kRows, m0 = (int)(block - slab * blocks) * COLS;  // (CTAs of the same rows of W are neighbours)
  const int chunks = (a.K + kChunk - 1) / kChunk, workers = (int)a.split * kWarps, me = (int)rank * kWarps + warp;
  const int c0 = (int)((long long)chunks * me / workers), c1 = (int)((long long)chunks * (me + 1) / workers);
  const uint32_t base = smem_addr(ring[warp]);
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
      next += i == kTiles - 1 ? kChunk / 2 - (2 * kTiles - 2) * by8 : 2 * by8;
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
  const uint16_t* xrow[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) xrow[nt] = a.x + min(m0 + nt * 8 + g, a.M - 1) * a.ldx;
  auto load_x = [&](int c, uint4 (&v)[NT][4]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int k = c * kChunk + w / VEC * 32 * VEC + t * 8 * VEC + w % VEC * 8;
        v[nt][w] = __ldg(reinterpret_cast<const uint4*>(xrow[nt] + (VEC == 4 ? k : min(k, a.K - 8))));
      }
  };

  float total[kTiles][NT][4] = {};
  uint4 xn[NT][4];
  uint16_t sn[Q][2];
  uint8_t zn[Q][2];
#pragma unroll
  for (int st = 0; st < kAhead; ++st) issue(c0 + st / kTiles, st % kTiles, st);
  load_x(min(c0, chunks - 1), xn);
  load_scales(min(c0, chunks - 1), sn, zn);
  int slot = 0;  // of the chunk's first step
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    uint32_t b[NT][4][4], sz[Q][2];  // (a scale in the high half, its zero in the low byte)
    float undo[NT][2];  // x's power of two, of the lane's columns
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t top = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (VEC < 4 && c * kChunk + w / VEC * 32 * VEC + t * 8 * VEC >= a.K) xn[nt][w] = make_uint4(0, 0, 0, 0);
        const uint4 v = xn[nt][w];
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                     __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
      }
      top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 2));
      const int ex = (int)(max(top & 0xffffu, top >> 16) >> 7);  // biased exponent of the largest value
      // the largest value's exponent becomes 30; the 1/16 of the high codes takes four more
      const uint32_t low = (uint32_t)max(ex - 30, 0) * 0x00800080u, low16 = low + 4 * 0x00800080u;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint4 v = xn[nt][w];
        b[nt][w][0] = to_f16x2(__byte_perm(v.x, v.z, 0x5410), low);
        b[nt][w][1] = to_f16x2(__byte_perm(v.x, v.z, 0x7632), low16);
        b[nt][w][2] = to_f16x2(__byte_perm(v.y, v.w, 0x5410), low);
        b[nt][w][3] = to_f16x2(__byte_perm(v.y, v.w, 0x7632), low16);
      }
      // 2^(low - 112): fp16's exponents are biased by 15, bf16's by 127; NaN for a row that is not finite
      const int e = max(ex - 30, 0) + 15;
      const float f = ex == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)e << 23);
#pragma unroll
      for (int j = 0; j < 2; ++j) undo[nt][j] = __shfl_sync(kFull, f, (2 * t + j) * 4);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int r = 0; r < 2; ++r) sz[q][r] = (uint32_t)sn[q][r] << 16 | (a.zeros ? zn[q][r] : 8u);
    load_x(min(c + 1, c1 - 1), xn);
    load_scales(min(c + 1, c1 - 1), sn, zn);
    const uint32_t here = base + g * kPitch + t * VEC * 4;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      issue(c + (i + kAhead) / kTiles, (i + kAhead) % kTiles, (slot + i + kAhead) & (kStages - 1));
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
      __syncwarp();
      uint32_t u[4], v[4];
#pragma unroll
      for (int l = 0; l < L; ++l) {
        const uint32_t p = here + ((slot + i) & (kStages - 1)) * kStageBytes + l * VEC * 16;
        if constexpr (VEC == 4) {
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(p) : "memory");
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(p + 8 * kPitch) : "memory");
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
        float acc[NT][4] = {}, acc2[NT][4] = {};  // (two chains of products)
#pragma unroll
        for (int w = l * VEC; w < (l + 1) * VEC; ++w) {
          const uint32_t a0 = low_codes(u[w], z0), a1 = low_codes(v[w], z1), a2 = high_codes(u[w], y0), a3 = high_codes(v[w], y1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt], a0, a1, a2, a3, b[nt][w][0], b[nt][w][1]);
          const uint32_t u8 = u[w] >> 8, v8 = v[w] >> 8;
          const uint32_t d0 = low_codes(u8, z0), d1 = low_codes(v8, z1), d2 = high_codes(u8, y0), d3 = high_codes(v8, y1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(acc2[nt], d0, d1, d2, d3, b[nt][w][2], b[nt][w][3]);
        }
        const float s0 = bf16_hi(sz0), s1 = bf16_hi(sz1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            total[i][nt][e] =
                __fmaf_rn(e < 2 ? s0 : s1, (acc[nt][e] + acc2[nt][e]) * undo[nt][e & 1], total[i][nt][e]);
      }
      __syncwarp();
    }
    slot = (slot + kTiles) & (kStages - 1);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // (the ring is read no more)
  const int cols = min(COLS, a.M - m0);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (nt * 8 + 2 * t + j < cols) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          red[warp][nt * 8 + 2 * t + j][i * 16 + g] = total[i][nt][j];
          red[warp][nt * 8 + 2 * t + j][i * 16 + g + 8] = total[i][nt][2 + j];
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
  // the CTAs of a cluster add their sums in the order of their ranks, each for a part of the outputs
  for (int x = (int)rank * kThreads + tid; x < kRows * cols; x += (int)a.split * kThreads) {
    const int r = x % kRows, col = x / kRows, n = n0 + r;
    const long long m = m0 + col;
    float z[1] = {0.f};
    if (a.split > 1) {
      for (unsigned q = 0; q < a.split; ++q) z[0] += tc::ld_cluster(tc::cluster_addr(&part[col][r], q));
    } else {
      z[0] = part[col][r];
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
  if (a.split > 1) tc::cluster_sync();  // (no CTA leaves while its sums are read)
}

template <int NT, int VEC>
cudaError_t launch(Args a, void* stream) {
  // as many CTAs as the card holds at once, as long as a warp keeps a chunk of k
  constexpr int rows = Shape<NT>::kRows;
  const long long slabs = ((a.N + rows - 1LL) / rows) * ((a.M + 8 * NT - 1LL) / (8 * NT));
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const long long fit = (long long)tc::num_sms() * Shape<NT>::kCtas / slabs;
  a.split = (unsigned)(fit < 1 ? 1 : fit > 8 ? 8 : fit);
  while (a.split > 1 && chunks < (int)a.split * kWarps) --a.split;
  if (slabs * a.split > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(slabs * a.split), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, rows_kernel<NT, VEC>, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int NT>
cudaError_t by_group(const Args& a, int group, void* stream) {
  return group == 128 ? launch<NT, 4>(a, stream) : group == 64 ? launch<NT, 2>(a, stream) : launch<NT, 1>(a, stream);
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
  const cudaError_t e = L.M <= 8 ? w4::by_group<1>(a, L.group, L.stream) : w4::by_group<2>(a, L.group, L.stream);
  if (e == cudaSuccess) return SV_OK;
  *err = std::string("linear_w4 launch: ") + cudaGetErrorString(e);
  return SV_ERR_CUDA;
}

}  // namespace sv
