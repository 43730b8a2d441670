// The matrix product of few rows with 4-bit weights, group scales, and the
// epilogue of sv_linear:
//
//   z[m][n] = sum_g s[n][g] sum_{k in g} (c[n][k] - zero[n][g]) x[m][k] + bias[n]
//   out[m][n] = act(z[m][n]) + residual[m][n]
//
// Bound by the bytes of W.  A code less its zero is an integer of -15 .. 15, which bf16 holds
// exactly: the tensor cores sum a group's products in float32 and the scale multiplies that
// sum, so no weight is rounded.  W is the 16-row side of mma.m16n8k16 and x the 8-column side.
// A lane's operands of a k step are any four codes of a row if x's values follow the same
// order, so a word of 8 codes (k .. k + 7, as it lies in memory) becomes two steps' operands in
// registers, 11 instructions for 8 codes: (w >> 4 j) & 0x000f000f | 0x43004300 is the pair of
// bf16 128 + c, from which 128 + zero is subtracted.  Eight warps of a CTA share 16 or 32 rows
// of W and take 128 k in turn; their sums meet in shared memory in a fixed order.
#include <atomic>
#include <cstdint>

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
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// codes 4 j (low half) and 4 j + 16 of a word, less the zero
template <int J>
__device__ __forceinline__ uint32_t codes(uint32_t w, uint32_t zero) {
  return sub_bf16x2((w >> (4 * J) & 0x000f000fu) | 0x43004300u, zero);
}

// What a warp holds of a chunk: 4 words of each of its lane's rows, their scale and zero.
template <int MT, int VEC>
struct Step {
  uint32_t w[2 * MT][4];
  uint32_t sz[2 * MT];  // scale in the high half, zero in the low byte
};

// VEC words (VEC * 32 k: a group) a load.
template <int MT, int VEC>
__device__ __forceinline__ void load_step(Step<MT, VEC>& s, const Args& a, const uint8_t* const (&row)[2 * MT],
                                          const long long (&srow)[2 * MT], int c, int t) {
#pragma unroll
  for (int r = 0; r < 2 * MT; ++r) {
#pragma unroll
    for (int l = 0; l < 4 / VEC; ++l) {
      const int k = c * kChunk + l * 32 * VEC + t * 8 * VEC;
      uint32_t* w = s.w[r] + l * VEC;
      if (k < a.K) {
        if constexpr (VEC == 4) {
          const uint4 v = __ldcs(reinterpret_cast<const uint4*>(row[r] + k / 2));
          w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (VEC == 2) {
          const uint2 v = __ldcs(reinterpret_cast<const uint2*>(row[r] + k / 2));
          w[0] = v.x, w[1] = v.y;
        } else {
          w[0] = __ldcs(reinterpret_cast<const uint32_t*>(row[r] + k / 2));
        }
      } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) w[v] = 0;
      }
    }
    // the lane's group of the chunk; the others' come by shuffle
    const int group = c * (4 / VEC) + (t & (4 / VEC - 1));
    uint32_t sz = 8;
    if (group < a.groups) {
      sz = (uint32_t)__ldg(a.scales + srow[r] + group) << 16;
      sz |= a.zeros ? __ldg(a.zeros + srow[r] + group) : 8;
    }
    s.sz[r] = sz;
  }
}

template <int MT, int NT, int VEC>
__global__ void __launch_bounds__(kThreads, 2) rows_kernel(const __grid_constant__ Args a) {
  constexpr int ROWS = 16 * MT, COLS = 8 * NT;
  __shared__ float red[kWarps][COLS][ROWS + 4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  pdl_wait();
  const int blocks = (a.M + COLS - 1) / COLS, tile = (int)(blockIdx.x / blocks);
  const int n0 = tile * ROWS, m0 = (int)(blockIdx.x - tile * blocks) * COLS;  // (CTAs of a tile are neighbours)
  const uint8_t* row[2 * MT];
  long long srow[2 * MT];
#pragma unroll
  for (int r = 0; r < 2 * MT; ++r) {
    const int n = min(n0 + g + 8 * r, a.N - 1);
    row[r] = a.W + n * a.ldw;
    srow[r] = (long long)n * a.groups;
  }
  const uint16_t* xrow[NT];
  bool has[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    has[nt] = m0 + nt * 8 + g < a.M;
    xrow[nt] = a.x + (has[nt] ? m0 + nt * 8 + g : 0) * a.ldx;
  }
  const int chunks = (a.K + kChunk - 1) / kChunk;
  float total[MT][NT][4] = {};

  auto consume = [&](const Step<MT, VEC>& s, int c) {
    float acc[MT][NT][4] = {};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int l = w / VEC, k = c * kChunk + l * 32 * VEC + t * 8 * VEC + (w % VEC) * 8;
      uint32_t b[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (has[nt] && k < a.K) v = __ldg(reinterpret_cast<const uint4*>(xrow[nt] + k));
        b[nt][0] = __byte_perm(v.x, v.z, 0x5410);
        b[nt][1] = __byte_perm(v.x, v.z, 0x7632);
        b[nt][2] = __byte_perm(v.y, v.w, 0x5410);
        b[nt][3] = __byte_perm(v.y, v.w, 0x7632);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const uint32_t sz0 = VEC == 4 ? s.sz[2 * mt] : __shfl_sync(kFull, s.sz[2 * mt], (lane & ~3) + l);
        const uint32_t sz1 = VEC == 4 ? s.sz[2 * mt + 1] : __shfl_sync(kFull, s.sz[2 * mt + 1], (lane & ~3) + l);
        const uint32_t z0 = 0x43004300u + (sz0 & 255u) * 0x10001u, z1 = 0x43004300u + (sz1 & 255u) * 0x10001u;
        const uint32_t u = s.w[2 * mt][w], v = s.w[2 * mt + 1][w];
        const uint32_t a0 = codes<0>(u, z0), a1 = codes<0>(v, z1), a2 = codes<1>(u, z0), a3 = codes<1>(v, z1);
        const uint32_t c0 = codes<2>(u, z0), c1 = codes<2>(v, z1), c2 = codes<3>(u, z0), c3 = codes<3>(v, z1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16(acc[mt][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16(acc[mt][nt], c0, c1, c2, c3, b[nt][2], b[nt][3]);
        if ((w + 1) % VEC == 0) {  // the group is complete
          const float s0 = bf16_hi(sz0), s1 = bf16_hi(sz1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              total[mt][nt][e] = __fmaf_rn(e < 2 ? s0 : s1, acc[mt][nt][e], total[mt][nt][e]);
              acc[mt][nt][e] = 0.f;
            }
        }
      }
    }
  };

  Step<MT, VEC> s0, s1;
  int c = warp;
  if (c < chunks) load_step<MT, VEC>(s0, a, row, srow, c, t);
  if (c + kWarps < chunks) load_step<MT, VEC>(s1, a, row, srow, c + kWarps, t);
  for (; c < chunks; c += 2 * kWarps) {
    consume(s0, c);
    if (c + 2 * kWarps < chunks) load_step<MT, VEC>(s0, a, row, srow, c + 2 * kWarps, t);
    if (c + kWarps < chunks) {
      consume(s1, c + kWarps);
      if (c + 3 * kWarps < chunks) load_step<MT, VEC>(s1, a, row, srow, c + 3 * kWarps, t);
    }
  }

#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        red[warp][nt * 8 + 2 * t + (e & 1)][mt * 16 + g + 8 * (e >> 1)] = total[mt][nt][e];
  __syncthreads();
  for (int x = tid; x < ROWS * COLS; x += kThreads) {
    const int r = x % ROWS, col = x / ROWS, n = n0 + r;
    const long long m = m0 + col;
    if (n >= a.N || m >= a.M) continue;
    float z[1] = {0.f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) z[0] += red[w][col][r];
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

template <int MT, int NT, int VEC>
cudaError_t launch(const Args& a, void* stream) {
  cudaLaunchConfig_t cfg = {};
  const long long ctas = ((a.N + 16 * MT - 1LL) / (16 * MT)) * ((a.M + 8 * NT - 1LL) / (8 * NT));
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, rows_kernel<MT, NT, VEC>, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int MT, int NT>
cudaError_t by_group(const Args& a, int group, void* stream) {
  return group == 128 ? launch<MT, NT, 4>(a, stream) : group == 64 ? launch<MT, NT, 2>(a, stream) : launch<MT, NT, 1>(a, stream);
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
  // 32 rows of W a CTA halve the reads of x; 16 where 32 would leave SMs without a CTA
  const bool wide = (L.N + 31) / 32 >= 2 * tc::num_sms();
  cudaError_t e;
  if (L.M <= 8) e = wide ? w4::by_group<2, 1>(a, L.group, L.stream) : w4::by_group<1, 1>(a, L.group, L.stream);
  else e = wide ? w4::by_group<2, 2>(a, L.group, L.stream) : w4::by_group<1, 2>(a, L.group, L.stream);
  if (e == cudaSuccess) return SV_OK;
  *err = std::string("linear_w4 launch: ") + cudaGetErrorString(e);
  return SV_ERR_CUDA;
}

}  // namespace sv
