// out = act(sx sw x W^T + bias) + residual: one 16 x 16 tile of outputs per
// CTA, operands staged in shared memory as float32.
#include <cstdint>

#include <cuda_fp8.h>

#include "sv_common.cuh"
#include "sv_internal.h"

namespace sv {
namespace lin {

struct Args {
  const void* x;
  long long ldx;
  const float* sx;
  const void* W;
  long long ldw;
  const float* sw;
  const uint16_t* bias;
  const void* res;
  long long ldr;
  void* out;
  long long ldo;
  int act, out_f32, M, N, K;
};

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case SV_ACT_RELU: return z < 0.f ? 0.f : z;  // (a NaN stays)
    case SV_ACT_SILU: return z / (1.f + __expf(-z));
    case SV_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    case SV_ACT_GELU_TANH:
      return 0.5f * z * (1.f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
    default: return z;
  }
}

__device__ __forceinline__ float value(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float value(const __nv_fp8_e4m3* p) { return float(*p); }

template <typename T>
__global__ void __launch_bounds__(256) linear_kernel(const Args a) {
  __shared__ float xs[16][17], ws[16][17];
  pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const long long tiles_n = (a.N + 15) / 16;
  const long long m0 = blockIdx.x / tiles_n * 16, n0 = blockIdx.x % tiles_n * 16;
  const T* x = static_cast<const T*>(a.x);
  const T* W = static_cast<const T*>(a.W);
  float acc = 0.f;
  for (int k0 = 0; k0 < a.K; k0 += 16) {
    const int k = k0 + tx;
    xs[ty][tx] = m0 + ty < a.M && k < a.K ? value(x + (m0 + ty) * a.ldx + k) : 0.f;
    ws[ty][tx] = n0 + ty < a.N && k < a.K ? value(W + (n0 + ty) * a.ldw + k) : 0.f;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 16; ++j) acc = __fmaf_rn(xs[ty][j], ws[tx][j], acc);
    __syncthreads();
  }
  const long long m = m0 + ty, n = n0 + tx;
  if (m >= a.M || n >= a.N) return;
  float z = acc * (a.sx ? a.sx[m] : 1.f) * (a.sw ? a.sw[n] : 1.f);
  if (a.bias) z += value(a.bias + n);
  z = activate(z, a.act);
  if (a.out_f32) {
    if (a.res) z += static_cast<const float*>(a.res)[m * a.ldr + n];
    static_cast<float*>(a.out)[m * a.ldo + n] = z;
  } else {
    if (a.res) z += value(static_cast<const uint16_t*>(a.res) + m * a.ldr + n);
    static_cast<uint16_t*>(a.out)[m * a.ldo + n] = __bfloat16_as_ushort(__float2bfloat16_rn(z));
  }
}

}  // namespace lin

int linear_launch(const LinearLaunch& L, std::string* err) {
  const lin::Args a = {L.x, L.ldx, L.x_scale, L.W, L.ldw, L.w_scale, static_cast<const uint16_t*>(L.bias),
                       L.residual, L.ldr, L.out, L.ldo, L.act, L.out_dtype == SV_F32 ? 1 : 0, L.M, L.N, L.K};
  const long long tiles = ((L.M + 15LL) / 16) * ((L.N + 15LL) / 16);
  if (tiles > 0x7fffffffLL) {
    *err = "M * N too large";
    return SV_ERR_SHAPE;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles, 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(L.stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = L.in_dtype == SV_BF16
                            ? cudaLaunchKernelEx(&cfg, lin::linear_kernel<uint16_t>, a)
                            : cudaLaunchKernelEx(&cfg, lin::linear_kernel<__nv_fp8_e4m3>, a);
  if (e != cudaSuccess) {
    *err = std::string("linear launch: ") + cudaGetErrorString(e);
    return SV_ERR_CUDA;
  }
  return SV_OK;
}

}  // namespace sv
