// Tensor-core, TMA and tensor-memory helpers (sm_103a inline PTX) of the layer
// operators, and the host side of their tensor maps.
#pragma once

#include <cuda.h>  // CUtensorMap and the encoder's signature (resolved at run time)

#include <atomic>
#include <cstdint>
#include <string>

#include "sv_common.cuh"
#include "sv_internal.h"

namespace sv {
namespace tc {

// Instruction descriptor: float32 accumulator (bits 4-5), operand formats (bits
// 7-9, 10-12: 1 bf16 of kind::f16, 0 e4m3 of kind::f8f6f4), B N-major at bit 16,
// N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc(bool f8, bool b_nmajor, int m, int n) {
  return (1u << 4) | (f8 ? 0u : (1u << 7) | (1u << 10)) | (b_nmajor ? 1u << 16 : 0u) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Shared-memory matrix descriptor, 128-byte swizzle: start address, leading and
// stride byte offsets (>> 4), version 1 (bit 46), swizzle 128 B (bits 61-63).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D (tensor memory) = A B (+ D if acc) with A, B from shared memory
template <int G, bool F8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  if constexpr (F8) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::%5.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"(acc), "n"(G)
                 : "memory");
  } else {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::%5.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"(acc), "n"(G)
                 : "memory");
  }
}

// The same for bf16, and with A (bf16 pairs, one row per lane) from tensor memory,
// with descriptors whose high word is kDescHigh given by their low words: in a loop of small products the issuing thread's arithmetic
// counts (a product of 128 x 128 x 16 takes 64 clocks).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride 1024, version 1, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); }
__device__ __forceinline__ void mma_low(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %4, 0;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n"
               " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}" ::"r"(d),
               "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescHigh)
               : "memory");
}
__device__ __forceinline__ void mma_ts_low(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %4, 0;\n mov.b64 y, {%2, %5};\n"
               " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}" ::"r"(d),
               "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescHigh)
               : "memory");
}

// one arrival on `bar` (a shared::cluster address) once every tcgen05 operation
// that this thread issued is done
template <int G>
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::%1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar), "n"(G)
               : "memory");
}

template <int G>
__device__ __forceinline__ void alloc(uint32_t* to, uint32_t columns) {  // one whole warp
  asm volatile("tcgen05.alloc.cta_group::%2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(to)),
               "r"(columns), "n"(G)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::%0.sync.aligned;" ::"n"(G) : "memory");
}
template <int G>
__device__ __forceinline__ void dealloc(uint32_t base, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::%2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns), "n"(G) : "memory");
}

// 32 (16) consecutive 32-bit columns of this warp's 32 lanes; the registers are
// valid behind ld_wait(), which names them so that no use moves in front of it.
#define SV_R16(c, v, o)                                                                                       \
  c(v[o]), c(v[o + 1]), c(v[o + 2]), c(v[o + 3]), c(v[o + 4]), c(v[o + 5]), c(v[o + 6]), c(v[o + 7]), c(v[o + 8]), \
      c(v[o + 9]), c(v[o + 10]), c(v[o + 11]), c(v[o + 12]), c(v[o + 13]), c(v[o + 14]), c(v[o + 15])
#define SV_OUT(x) "=r"(x)
#define SV_INOUT(x) "+r"(x)
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : SV_R16(SV_OUT, v, 0), SV_R16(SV_OUT, v, 16)
      : "r"(taddr));
}
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : SV_R16(SV_OUT, v, 0)
      : "r"(taddr));
}
__device__ __forceinline__ void ld_wait(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : SV_R16(SV_INOUT, v, 0)::"memory");
  asm volatile("" : SV_R16(SV_INOUT, v, 16));
}
__device__ __forceinline__ void ld_wait(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : SV_R16(SV_INOUT, v, 0)::"memory");
}
#undef SV_R16
#undef SV_OUT
#undef SV_INOUT

// Columns back into tensor memory; st_wait() before anyone reads them.
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// The address of `p` (in this CTA's shared memory) in the CTA of cluster rank `rank`.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}

// Box of a 2-D tensor map at (x, y) into shared memory, counted on `bar`.
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
// The same, counted on a barrier of either CTA of a pair (shared::cluster address).
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Box of a 4-D tensor map.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Arrival on a barrier of another CTA of the cluster, releasing this thread's
// earlier operations at cluster scope.
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Bounded waits: for the completion of the phase of this parity, at most about a
// second (kWaitClocks).  Without a suspend-time hint: a thread that the hint put to
// sleep woke up to a thousand clocks late.
constexpr long long kWaitClocks = 2000000000LL;
template <bool CLUSTER>
__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (CLUSTER)
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
  else
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok)
                 : "r"(smem_addr(bar)), "r"(parity)
                 : "memory");
  return ok != 0;
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, long long clocks = kWaitClocks) {
  if (try_wait<CLUSTER>(bar, parity)) return true;
  const long long start = clock64();
  while (clock64() - start < clocks)
    if (try_wait<CLUSTER>(bar, parity)) return true;
  return false;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encoder(std::string* err) {
  static std::atomic<EncodeTiledFn> found{nullptr};
  EncodeTiledFn f = found.load(std::memory_order_acquire);
  if (!f) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) {
      *err = std::string("cuTensorMapEncodeTiled is not available: ") + cudaGetErrorString(e);
      return nullptr;
    }
    f = reinterpret_cast<EncodeTiledFn>(fn);
    found.store(f, std::memory_order_release);
  }
  return f;
}

// Rows of `inner` elements (bf16, or bytes for 8-bit types) `row_bytes` apart;
// boxes of 128 bytes x box_rows, 128-byte swizzle, zeros outside.
inline bool make_map(EncodeTiledFn enc, CUtensorMap* map, bool bytes, const void* base, uint64_t inner, uint64_t rows,
                     uint64_t row_bytes, uint32_t box_rows, std::string* err) {
  const cuuint64_t dims[2] = {inner, rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {bytes ? 128u : 64u, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                         const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    *err = "cuTensorMapEncodeTiled failed with CUresult " + std::to_string((int)r);
    return false;
  }
  return true;
}

// SM count of the current device (148 if it cannot be read).
inline int num_sms() {
  static std::atomic<int> cache[kMaxDevices];
  const int d = current_device();
  if (d < 0) return 148;
  int n = cache[d].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d) != cudaSuccess || n < 1) n = 148;
    cache[d].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace tc
}  // namespace sv
