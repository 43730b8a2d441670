// Attention of a round's query positions over a shared prefix and the paged
// cache of each sequence's own tokens: one warp per query row, one pass with
// the running maximum and sum of the softmax.
#include <cstdint>

#include "sv_common.cuh"
#include "sv_internal.h"

namespace sv {
namespace att {

__global__ void clear_kernel(uint32_t* flags) {
  pdl_wait();
  *flags = 0u;
}

template <int D>
__global__ void __launch_bounds__(256) rows_kernel(const AttentionLaunch a, uint32_t* flags) {
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int Q = a.K + 1, G = a.Hq / a.Hkv;
  if (row >= (long long)a.B * Q * a.Hq) return;
  const int h = (int)(row % a.Hq), i = (int)(row / a.Hq % Q), b = (int)(row / a.Hq / Q);
  const int k = a.kpr ? a.kpr[b] : a.K, len = a.lens[b];
  uint32_t bad = 0;
  if (k < 0 || k > a.K) bad = SV_FLAG_BAD_K;
  else if (i > k) return;
  else if (len < 0 || (long long)len + k > (long long)a.max_pages * a.page_size) bad = SV_FLAG_BAD_N;
  const uint16_t* K_ = static_cast<const uint16_t*>(a.k) + (h / G) * a.head;
  const uint16_t* V_ = static_cast<const uint16_t*>(a.v) + (h / G) * a.head;
  constexpr int E = D / 32;
  float q[E], o[E], m = -INFINITY, l = 0.f;
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + b * a.q_seq + i * a.q_pos + h * a.q_head + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float((uint32_t)qp[e] << 16);
    o[e] = 0.f;
  }
  const int P = a.prefix_len;
  const int total = bad ? 0 : P + len + k;  // every key of the sequence: pages are checked for all of them
  for (int j = 0; j < total; ++j) {
    const int t = j < P ? j : j - P;
    const int page = j < P ? a.prefix_pages[t / a.page_size] : a.table[(long long)b * a.max_pages + t / a.page_size];
    if (page < 0 || page >= a.num_pages) {
      bad |= SV_FLAG_BAD_PAGE;
      continue;
    }
    if (j >= P + len + i) continue;
    const long long at = page * a.page + (t % a.page_size) * a.token + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * __uint_as_float((uint32_t)K_[at + e] << 16);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale;
    const float nm = s > m ? s : m;
    const float c = nm == -INFINITY ? 1.f : __expf(m - nm), p = nm == -INFINITY ? 0.f : __expf(s - nm);
    l = l * c + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * __uint_as_float((uint32_t)V_[at + e] << 16);
    m = nm;
  }
  uint16_t* op = static_cast<uint16_t*>(a.out) + b * a.o_seq + i * a.o_pos + h * a.o_head + lane * E;
  const float nan = __int_as_float(0x7fffffff);
#pragma unroll
  for (int e = 0; e < E; ++e)
    op[e] = __bfloat16_as_ushort(__float2bfloat16_rn(bad ? nan : (l == 0.f ? 0.f : o[e] / l)));
  if (a.lse && lane == 0) a.lse[row] = bad ? nan : (l == 0.f ? -INFINITY : m + logf(l));
  if (bad && lane == 0) atomicOr(flags, bad);
}

}  // namespace att

size_t attention_workspace_bytes(int, int, int, int, int, int, int) { return 256; }

int attention_launch(const AttentionLaunch& L, std::string* err) {
  cudaStream_t st = static_cast<cudaStream_t>(L.stream);
  uint32_t* flags = static_cast<uint32_t*>(L.workspace);
  att::clear_kernel<<<1, 1, 0, st>>>(flags);
  const long long rows = (long long)L.B * (L.K + 1) * L.Hq;
  const unsigned blocks = (unsigned)((rows + 7) / 8);
  if (L.D == 128)
    att::rows_kernel<128><<<blocks, 256, 0, st>>>(L, flags);
  else
    att::rows_kernel<64><<<blocks, 256, 0, st>>>(L, flags);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    *err = std::string("attention launch: ") + cudaGetErrorString(e);
    return SV_ERR_CUDA;
  }
  return SV_OK;
}

}  // namespace sv
