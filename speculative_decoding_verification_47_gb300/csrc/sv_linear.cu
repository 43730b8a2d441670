// The matrix product of a layer with bias, activation and residual in its
// epilogue, on the 5th-generation tensor cores:
//
//   z[m][n] = sx[m] sw[n] sum_k x[m][k] W[n][k] + bias[n]
//   out[m][n] = act(z[m][n]) + residual[m][n]
//
// x and W are bf16 or e4m3, K contiguous in both: both operands are K-major,
// one 128-byte swizzle row (64 bf16 or 128 e4m3 values) per k block, so the two
// types share every tile and differ in the instruction alone.  Sums are float32
// in tensor memory; the scales, which leave the sum, come in the epilogue.
//
// Two kernels:
//  * rows_kernel (few rows of x): W is the MMA's 128-row operand and x its N
//    side, 16 to 128 columns.  Bound by the bytes of W.  A cluster splits K and
//    adds its partial sums through distributed shared memory in rank order.
//  * pair_kernel (more rows): persistent CTA pairs, tiles of MS x 256 rows by BN
//    columns with cta_group::2, each CTA staging its rows of x and half of W's.
#include <cstdint>
#include <string>

#include "sv_act.cuh"
#include "sv_tc.cuh"

namespace sv {
namespace lin {

struct Epilogue {
  const float* sx;
  const float* sw;
  const uint16_t* bias;
  const void* res;
  long long ldr;
  void* out;
  long long ldo;
  int act, out_f32, M, N;
  int vec;  // rows of out and residual start on 16-byte boundaries
  uint32_t tries;  // of a wait for a sum
};

__device__ __forceinline__ float bf16(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// One output from its sum and its residual.
__device__ __forceinline__ void finish(const Epilogue& e, long long m, int n, float acc, float sw, float bias,
                                       float res) {
  float z[1] = {__fmaf_rn(acc, (e.sx ? e.sx[m] : 1.f) * sw, bias)};
  activate(z, e.act);
  if (e.res) z[0] += res;
  if (e.out_f32)
    static_cast<float*>(e.out)[m * e.ldo + n] = z[0];
  else
    static_cast<uint16_t*>(e.out)[m * e.ldo + n] = __bfloat16_as_ushort(__float2bfloat16_rn(z[0]));
}

// The tensor cores add a product of one k step to the float32 accumulator by
// cutting, not rounding: over K = 16384 (bf16) a float32 result is off by 1.9e-5
// of its norm, sixty times the rounding sums' error.  Below a bf16 output that is
// nothing (2^-9); for a float32 one the accumulation is cut into kChunk k blocks
// (128 instructions, about 2e-6) whose sums are added with rounding.
constexpr int kChunk = 32;

// What a sum becomes whose wait ran out; every epilogue keeps it.
constexpr uint32_t kNan = 0x7fffffffu;

constexpr int kRowBytes = 128;       // a k block of one row
constexpr int kTile = 128 * kRowBytes;  // 128 rows of one k block

// ---------------------------------------------------------------------------
// Few rows of x: a tile is 128 rows of W by TM rows of x.
// ---------------------------------------------------------------------------
constexpr int kRowsThreads = 192;

template <int TM>
struct RowsShape {
  static constexpr int kStageBytes = kTile + TM * kRowBytes;
  static constexpr int kStages = 100 * 1024 / kStageBytes;  // two CTAs per SM
  static constexpr int kSmem = kStages * kStageBytes + 1024;
  static constexpr uint32_t kColumns = TM < 32 ? 32 : TM;
  static_assert(kStages * kStageBytes >= TM * 128 * 4, "the partial sums fit over the ring");
};

template <int TM, bool F8>
__global__ void __launch_bounds__(kRowsThreads, 2)
    rows_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const Epilogue e,
                int KB, int split, uint32_t* flags) {
  using S = RowsShape<TM>;
  constexpr uint32_t kId = tc::idesc(F8, false, 128, TM);
  constexpr int kElems = F8 ? 128 : 64;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages], done;
  __shared__ uint32_t tmem_base;
  __shared__ int issued, consumed, failed;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % split, tile = blockIdx.x / split, n0 = tile * 128;
  const int k_lo = (int)((long long)KB * rank / split), k_hi = (int)((long long)KB * (rank + 1) / split);
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    issued = consumed = failed = 0;
    fence_mbar_init();
    tc::prefetch_map(&tmX);
    tc::prefetch_map(&tmW);
    // W's first boxes into L2 while an earlier kernel of the stream may still run
    for (int k = k_lo; k < k_hi && k < k_lo + S::kStages; ++k) tc::tma_prefetch(&tmW, k * kElems, n0);
  }
  if (warp == 0) tc::alloc<1>(&tmem_base, S::kColumns);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_base;
  pdl_launch_dependents();  // (behind the allocation: a dependent cannot take this CTA's columns)
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      int g = 0;
      for (int k = k_lo; k < k_hi; ++k, ++g) {
        const int s = g % S::kStages, use = g / S::kStages;
        if (use > 0 && !mbar_wait_bounded(&empty[s], (uint32_t)((use - 1) & 1))) {
          failed = 1;
          break;
        }
        uint8_t* w = smem + s * S::kStageBytes;
        mbar_arrive_expect_tx(&full[s], (uint32_t)S::kStageBytes);
        tc::tma_load(w, &tmW, k * kElems, n0, &full[s]);
        tc::tma_load(w + kTile, &tmX, k * kElems, 0, &full[s]);
      }
      issued = g;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int g = 0;
      for (int k = k_lo; k < k_hi; ++k, ++g) {
        const int s = g % S::kStages;
        if (!mbar_wait_bounded(&full[s], (uint32_t)((g / S::kStages) & 1))) {
          failed = 1;
          break;
        }
        tc::fence_after();
        const uint32_t w = smem_addr(smem + s * S::kStageBytes);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          tc::mma<1, F8>(tmem, tc::desc_sw128(w + 32 * q, 16, 1024), tc::desc_sw128(w + kTile + 32 * q, 16, 1024), kId,
                         (g | q) != 0);
        tc::commit<1>(smem_addr(&empty[s]));
      }
      consumed = g;
      tc::commit<1>(smem_addr(&done));
    }
  }
  __syncwarp();
  // every thread: the accumulator is complete (so all loads have landed, too)
  if (!mbar_wait_bounded(&done, 0, e.tries)) failed = 1;
  tc::fence_after();
  __syncthreads();
  const bool lost = failed != 0;  // (the same in every thread)
  if (lost) {  // a wait ran out: copies and products on their way end first, and the tile is NaN
    if (tid == 0) {
      atomicOr(flags, SV_FLAG_TIMEOUT);
      for (int g = consumed; g < issued; ++g)
        (void)mbar_wait_bounded(&full[g % S::kStages], (uint32_t)((g / S::kStages) & 1), 64);
      (void)mbar_wait_bounded(&done, 0);
    }
    __syncthreads();
  }
  const int n = n0 + (warp & 3) * 32 + lane;
  const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  if (split == 1) {
    if (warp >= 2) {
      const float sw = e.sw && n < e.N ? e.sw[n] : 1.f, bias = e.bias && n < e.N ? bf16(e.bias + n) : 0.f;
#pragma unroll 1
      for (int c = 0; c < TM && c < e.M; c += 16) {
        float res[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const long long m = c + j;
          res[j] = 0.f;
          if (e.res && m < e.M && n < e.N)
            res[j] = e.out_f32 ? static_cast<const float*>(e.res)[m * e.ldr + n]
                               : bf16(static_cast<const uint16_t*>(e.res) + m * e.ldr + n);
        }
        uint32_t v[16];
        tc::ld16(lanes + c, v);
        tc::ld_wait(v);
        if (n < e.N) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < e.M) finish(e, c + j, n, __uint_as_float(lost ? kNan : v[j]), sw, bias, res[j]);
        }
      }
    }
  } else {
    float* part = reinterpret_cast<float*>(smem);  // [TM][128]
    if (warp >= 2) {
#pragma unroll 1
      for (int c = 0; c < TM && c < e.M; c += 16) {
        uint32_t v[16];
        tc::ld16(lanes + c, v);
        tc::ld_wait(v);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          part[(c + j) * 128 + (warp & 3) * 32 + lane] = __uint_as_float(lost ? kNan : v[j]);
      }
    }
    tc::cluster_sync();
    // each CTA adds its share of the tile over the ranks, in rank order; kAtOnce
    // outputs of a thread are in flight together (their residuals first)
    constexpr int kAtOnce = 2;
    const uint32_t base = smem_addr(part);
    const int nn = n0 + (tid & 63), step = split * (kRowsThreads / 64);  // a thread keeps two columns
    float sw[2], bias[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sw[h] = e.sw && nn + 64 * h < e.N ? e.sw[nn + 64 * h] : 1.f;
      bias[h] = e.bias && nn + 64 * h < e.N ? bf16(e.bias + nn + 64 * h) : 0.f;
    }
    for (int m = rank * (kRowsThreads / 64) + (tid >> 6); m < e.M; m += step * kAtOnce) {
      float acc[kAtOnce][2], res[kAtOnce][2];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const long long mm = m + i * step;
          acc[i][h] = res[i][h] = 0.f;
          if (e.res && mm < e.M && nn + 64 * h < e.N)
            res[i][h] = e.out_f32 ? static_cast<const float*>(e.res)[mm * e.ldr + nn + 64 * h]
                                  : bf16(static_cast<const uint16_t*>(e.res) + mm * e.ldr + nn + 64 * h);
        }
      float of[kAtOnce][8][2];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        uint32_t at;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(base + 4u * (m * 128 + (tid & 63))), "r"(r < split ? r : 0));
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            of[i][r][h] = r < split && m + i * step < e.M ? tc::ld_cluster(at + 4u * (i * step * 128 + 64 * h)) : 0.f;
      }
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) acc[i][h] += of[i][r][h];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (m + i * step < e.M)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (nn + 64 * h < e.N) finish(e, m + i * step, nn + 64 * h, acc[i][h], sw[h], bias[h], res[i][h]);
    }
    tc::cluster_sync();  // no CTA leaves while another reads its sums
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) tc::dealloc<1>(tmem, S::kColumns);
}

// ---------------------------------------------------------------------------
// More rows: pairs of CTAs.
// ---------------------------------------------------------------------------
constexpr int kEpiWarps = 8;
constexpr int kPairThreads = 64 + 32 * kEpiWarps;
constexpr int kPairRing = 12 * kTile;  // 192 KB
constexpr int kOutStride = 17;         // floats: a row of 16 and one against bank conflicts
constexpr int kPairSmem = kPairRing + kEpiWarps * 32 * kOutStride * 4 + 1024;
constexpr int kBand = 8;

template <int BN, int MS>
struct PairShape {
  static constexpr int kStageBytes = MS * kTile + BN / 2 * kRowBytes;
  static constexpr int kStages = kPairRing / kStageBytes;  // 4 (512 x 256) to 8 (256 x 128)
  static constexpr int kBufs = 2 / MS;
};

// A chunk of W columns of this warp's 32 rows (one per lane, from row
// m on), in two steps: the residual is asked for before the accumulator is waited
// for.  Rows on 16-byte boundaries: every lane reads and writes its own row in
// 16-byte words, whole 32-byte sectors.
template <int W>
struct RowChunk {
  uint4 r[W / 4];  // (half of them for bf16)

  __device__ __forceinline__ void ask(const Epilogue& e, long long m, int n) {
    if (!e.res || m >= e.M) return;
    if (e.out_f32) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(e.res) + m * e.ldr + n);
#pragma unroll
      for (int q = 0; q < W / 4; ++q) r[q] = p[q];
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(e.res) + m * e.ldr + n);
#pragma unroll
      for (int q = 0; q < W / 8; ++q) r[q] = p[q];
    }
  }
  __device__ __forceinline__ void put(const Epilogue& e, long long m, int n, float (&z)[W]) const {
    if (m >= e.M) return;
    if (e.out_f32) {
      uint4* o = reinterpret_cast<uint4*>(static_cast<float*>(e.out) + m * e.ldo + n);
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        if (e.res) {
          z[4 * q] += __uint_as_float(r[q].x);
          z[4 * q + 1] += __uint_as_float(r[q].y);
          z[4 * q + 2] += __uint_as_float(r[q].z);
          z[4 * q + 3] += __uint_as_float(r[q].w);
        }
        o[q] = make_uint4(__float_as_uint(z[4 * q]), __float_as_uint(z[4 * q + 1]), __float_as_uint(z[4 * q + 2]),
                          __float_as_uint(z[4 * q + 3]));
      }
    } else {
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(e.out) + m * e.ldo + n);
#pragma unroll
      for (int q = 0; q < W / 8; ++q) {
        if (e.res) {
          const uint32_t w[4] = {r[q].x, r[q].y, r[q].z, r[q].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            z[8 * q + 2 * j] += bf16_lo(w[j]);
            z[8 * q + 2 * j + 1] += bf16_hi(w[j]);
          }
        }
        o[q] = make_uint4(tc::pack_bf16x2(z[8 * q], z[8 * q + 1]), tc::pack_bf16x2(z[8 * q + 2], z[8 * q + 3]),
                          tc::pack_bf16x2(z[8 * q + 4], z[8 * q + 5]), tc::pack_bf16x2(z[8 * q + 6], z[8 * q + 7]));
      }
    }
  }
};

// Any other alignment, and a tile's ragged end: 16 columns of this warp's 32 rows,
// which the lanes left in shared memory (`t`), two rows at a time with a lane per
// column, so that a store still covers whole runs of a row.  o, r: this lane's
// first element, `rows` rows above the matrix's end.
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ void narrow(float* p, float v) { *p = v; }
__device__ __forceinline__ void narrow(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

template <typename T>
__device__ __noinline__ void put_by_columns(T* o, long long ldo, const T* r, long long ldr, int rows, const float* t) {
  const int lane = threadIdx.x & 31;
  t += (lane >> 4) * kOutStride + (lane & 15);
#pragma unroll
  for (int h = 0; h < 32; h += 8) {
    float a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = t[(h + 2 * i) * kOutStride];
      if (r) {
        if (h + 2 * i < rows) a[i] += widen(*r);
        r += 2 * ldr;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (h + 2 * i < rows) narrow(o, a[i]);
      o += 2 * ldo;
    }
  }
}

// 16 columns from n on of this warp's rows: accumulator, scales, bias, activation,
// residual, store.  rc holds the residual, if the rows are whole 16-byte words.
__device__ __forceinline__ void chunk(const Epilogue& e, uint32_t at, long long m0, int n, float sx, const float* sw,
                                      const float* bias, bool rows, const RowChunk<16>& rc, float* t) {
  const long long m = m0 + (threadIdx.x & 31);
  constexpr int W = 16;
  uint32_t v[W];
  tc::ld16(at, v);
  tc::ld_wait(v);
  float z[W];
#pragma unroll
  for (int j = 0; j < W; ++j) z[j] = __fmaf_rn(__uint_as_float(v[j]), sx * sw[j], bias[j]);
  activate(z, e.act);
  if (rows) {
    rc.put(e, m, n, z);
  } else {
    __syncwarp();  // (the last chunk is read)
#pragma unroll
    for (int j = 0; j < 16; ++j) t[(threadIdx.x & 31) * kOutStride + j] = z[j];
    __syncwarp();
    const int nl = n + (threadIdx.x & 15);
    const long long ml = m0 + ((threadIdx.x >> 4) & 1);
    const int left = e.M - ml < 32 ? (int)(e.M - ml) : 32;
    if (nl < e.N) {
      if (e.out_f32)
        put_by_columns(static_cast<float*>(e.out) + ml * e.ldo + nl, e.ldo,
                       e.res ? static_cast<const float*>(e.res) + ml * e.ldr + nl : nullptr, e.ldr, left, t);
      else
        put_by_columns(static_cast<uint16_t*>(e.out) + ml * e.ldo + nl, e.ldo,
                       e.res ? static_cast<const uint16_t*>(e.res) + ml * e.ldr + nl : nullptr, e.ldr, left, t);
    }
  }
}

// LONG: at most kChunk k blocks are summed in tensor memory; the chunks' sums
// are added in registers (columns of a thread: BN / 2).
template <int BN, int MS, bool F8, bool LONG>
__global__ void __launch_bounds__(kPairThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const Epilogue e,
                int KB, uint32_t* flags) {
  using PS = PairShape<BN, MS>;
  constexpr int kSt = PS::kStages, kSB = PS::kStageBytes, NB = PS::kBufs, BH = BN / 2, TR = MS * 256;
  constexpr uint32_t kId = tc::idesc(F8, false, 256, BN);
  constexpr int kElems = F8 ? 128 : 64;
  static_assert(!LONG || MS == 1, "a thread keeps the sums of one sub-tile");
  constexpr uint32_t kTx = 2u * (uint32_t)(MS * kTile + BH * kRowBytes);  // both CTAs
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kSt], empty[kSt], accf[NB], acce[NB];
  __shared__ __align__(16) float col[2][2][BN];  // w_scale and bias of the tile's columns, by the tile's parity
  __shared__ uint32_t tmem_base;
  __shared__ int issued, consumed, failed;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t half = blockIdx.x & 1u;  // cluster rank; 0 is the pair's leader
  const int pid = (int)(blockIdx.x >> 1), npairs = (int)(gridDim.x >> 1);
  const int mt = (e.M + TR - 1) / TR, nt = (e.N + BN - 1) / BN;
  const long long tiles = (long long)mt * nt;
  // Tiles are numbered in bands of kBand row tiles, M-fastest inside a band, so
  // that the tiles in flight share both operands' blocks.
  const long long per_band = (long long)kBand * nt;
  auto place = [&](long long t, int& tm, int& tn) {
    const int bd = (int)(t / per_band), r0 = bd * kBand, h = mt - r0 < kBand ? mt - r0 : kBand;
    const long long in = t - bd * per_band;
    tm = r0 + (int)(in % h);
    tn = (int)(in / h);
  };
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (tid == 0) {
    for (int s = 0; s < kSt; ++s) {
      mbar_init(&full[s], 1);   // (the leader's: its arrival + both CTAs' bytes)
      mbar_init(&empty[s], 1);  // one commit from the leader's MMA thread
    }
    for (int b = 0; b < NB; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], 2 * kEpiWarps);  // (the leader's: the epilogue warps of both CTAs)
    }
    issued = consumed = failed = 0;
    fence_mbar_init();
    tc::prefetch_map(&tmX);
    tc::prefetch_map(&tmW);
  }
  if (warp == 0) tc::alloc<2>(&tmem_base, 512);
  tc::fence_before();
  tc::cluster_sync();  // both CTAs' barriers and columns exist before any remote use
  tc::fence_after();
  const uint32_t tmem = tmem_base;
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {  // ---- TMA producer (both CTAs): own rows of x, own half of W's ----
      int g = 0;
      bool ok = true;
      for (long long t = pid; t < tiles && ok; t += npairs) {
        int tm, tn;
        place(t, tm, tn);
        const int m0 = tm * TR + (int)half * 128, n0 = tn * BN + (int)half * BH;
        for (int kb = 0; kb < KB; ++kb, ++g) {
          const int s = g % kSt, use = g / kSt;
          if (use > 0 && !mbar_wait_bounded(&empty[s], (uint32_t)((use - 1) & 1))) {
            ok = false;
            break;
          }
          uint8_t* a = smem + s * kSB;
          if (half == 0) mbar_arrive_expect_tx(&full[s], kTx);
          const uint32_t fb = tc::cluster_addr(&full[s], 0u);
#pragma unroll
          for (int ms = 0; ms < MS; ++ms) tc::tma_load_pair(a + ms * kTile, &tmX, kb * kElems, m0 + ms * 256, fb);
          tc::tma_load_pair(a + MS * kTile, &tmW, kb * kElems, n0, fb);
        }
      }
      issued = g;
      if (!ok) failed = 1;
    }
  } else if (warp == 1) {
    if (lane == 0 && half == 0) {  // ---- MMA issuer: the leader only ----
      int g = 0, i = -1, b = 0;
      bool ok = true;
      for (long long t = pid; t < tiles && ok; t += npairs) {
        for (int kb = 0; kb < KB; ++kb, ++g) {
          const bool first = LONG ? kb % kChunk == 0 : kb == 0;
          if (first) {  // the next accumulator, once the epilogue has left it
            ++i;
            b = i % NB;
            if (i >= NB && !tc::wait_bounded<true>(&acce[b], (uint32_t)((i / NB - 1) & 1))) {
              ok = false;
              break;
            }
            tc::fence_after();
          }
          const int s = g % kSt;
          if (!mbar_wait_bounded(&full[s], (uint32_t)((g / kSt) & 1))) {
            ok = false;
            break;
          }
          tc::fence_after();
          const uint32_t a = smem_addr(smem + s * kSB), w = a + MS * kTile;
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int ms = 0; ms < MS; ++ms)
              tc::mma<2, F8>(tmem + (uint32_t)((b * MS + ms) * 256), tc::desc_sw128(a + ms * kTile + 32 * q, 16, 1024),
                             tc::desc_sw128(w + 32 * q, 16, 1024), kId, !first || q != 0);
          tc::commit<2>(tc::cluster_addr(&empty[s], 0u));  // the stage is free in both CTAs
          tc::commit<2>(tc::cluster_addr(&empty[s], 1u));
          if (kb == KB - 1 || (LONG && kb % kChunk == kChunk - 1)) {
            tc::commit<2>(tc::cluster_addr(&accf[b], 0u));
            tc::commit<2>(tc::cluster_addr(&accf[b], 1u));
          }
        }
      }
      consumed = g;
      if (!ok) failed = 1;
    }
  } else {
    // ---- epilogue: two warps per 32 tensor-memory lanes, half of the columns each ----
    const int lg = warp & 3, et = tid - 64, ch = (warp - 2) >> 2;
    float* stage = reinterpret_cast<float*>(smem + kPairRing) + (warp - 2) * 32 * kOutStride;
    int i = 0, turn = 0;
    bool lost = false;
    auto complete = [&](int b) {  // accumulator b, in its turn
      // a wait that runs out: on, since the other warps meet at the barrier below, but
      // with NaN and no further wait.  Nothing is released either, or a phase that this
      // warp did not see could end early and the products overwrite what others read.
      if (!lost && !__all_sync(0xffffffffu, mbar_wait_bounded(&accf[b], (uint32_t)((turn / NB) & 1), e.tries))) {
        failed = 1;
        lost = true;
      }
      tc::fence_after();
    };
    auto release = [&](int b) {
      tc::fence_before();
      __syncwarp();
      if (lane == 0 && !lost) tc::arrive_remote(tc::cluster_addr(&acce[b], 0u));
      ++turn;
    };
    for (long long t = pid; t < tiles; t += npairs, ++i) {
      int tm, tn;
      place(t, tm, tn);
      const int m0 = tm * TR + (int)half * 128, n0 = tn * BN;
      float(*c)[BN] = col[i & 1];
      if (et < BN) {
        const int n = n0 + et;
        c[0][et] = e.sw && n < e.N ? e.sw[n] : 1.f;
        c[1][et] = e.bias && n < e.N ? bf16(e.bias + n) : 0.f;
      }
      if (e.res) {  // the tile's residual into L2 while the products run
        const int es = e.out_f32 ? 4 : 2;
#pragma unroll 1
        for (int ms = 0; ms < MS; ++ms) {
          const long long m = m0 + ms * 256 + lg * 32 + lane;
          for (int k = ch * BH; m < e.M && k < (ch + 1) * BH && n0 + k < e.N; k += 128 / es)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(e.res) + (m * e.ldr + n0 + k) * es));
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
      int b = turn % NB;
      complete(b);
      if constexpr (LONG) {
        float sum[BH];
#pragma unroll
        for (int k = 0; k < BH; ++k) sum[k] = 0.f;
        for (int left = (KB + kChunk - 1) / kChunk - 1;; --left) {
          const uint32_t at = tmem + (uint32_t)(b * 256 + ch * BH) + ((uint32_t)(lg * 32) << 16);
#pragma unroll
          for (int k = 0; k < BH; k += 16) {
            uint32_t v[16];
            tc::ld16(at + k, v);
            tc::ld_wait(v);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              sum[k + j] += __uint_as_float(v[j]);
              v[j] = __float_as_uint(sum[k + j]);
            }
            if (left == 0) tc::st16(at + k, v);  // the whole sum, for the loop below
          }
          if (left == 0) break;
          release(b);
          b = turn % NB;
          complete(b);
        }
        tc::st_wait();
      }
#pragma unroll 1
      for (int ms = 0; ms < MS; ++ms) {
        const long long row0 = m0 + ms * 256 + lg * 32, m = row0 + lane;
        const uint32_t at = tmem + (uint32_t)((b * MS + ms) * 256) + ((uint32_t)(lg * 32) << 16);
        const float sx = lost ? __uint_as_float(kNan) : (e.sx && m < e.M ? e.sx[m] : 1.f);
        if (row0 >= e.M) break;
        RowChunk<16> rc, next;  // the residual is asked for one chunk ahead
        auto whole = [&](int k) { return e.vec && n0 + k + 16 <= e.N; };  // (the same in the whole warp)
        if (whole(ch * BH)) next.ask(e, m, n0 + ch * BH);
#pragma unroll 1
        for (int k = ch * BH; k < (ch + 1) * BH && n0 + k < e.N; k += 16) {
          rc = next;
          if (k + 16 < (ch + 1) * BH && whole(k + 16)) next.ask(e, m, n0 + k + 16);
          chunk(e, at + k, row0, n0 + k, sx, &c[0][k], &c[1][k], whole(k), rc, stage);
        }
      }
      release(b);
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (tid == 0 && failed) {
    atomicOr(flags, SV_FLAG_TIMEOUT);
    if (half == 0) {  // copies and products on their way end before the pair exits
      for (int g = consumed; g < issued; ++g) (void)mbar_wait_bounded(&full[g % kSt], (uint32_t)((g / kSt) & 1), 64);
      if (consumed > 0)
        (void)mbar_wait_bounded(&empty[(consumed - 1) % kSt], (uint32_t)(((consumed - 1) / kSt) & 1), 64);
    }
  }
  tc::cluster_sync();  // no CTA leaves while its peer may still signal or read it
  tc::fence_after();
  if (warp == 0) tc::dealloc<2>(tmem, 512);
}

// ---------------------------------------------------------------------------
// Too few tiles for the card: `split` pairs of one cluster share a tile's K.
// Each adds its k blocks in tensor memory, leaves the float32 sums in its ring
// (which is idle by then), and finishes 128 / split rows of its half of the tile
// over the pairs' sums, in rank order, read through distributed shared memory.
// One pair alone walks K at 0.32 us a block: 256 x 4096 x 4096 took 27.2 us.
// ---------------------------------------------------------------------------
template <int BN, bool F8>
__global__ void __launch_bounds__(kPairThreads, 1)
    split_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const Epilogue e,
                 int KB, int split, uint32_t* flags) {
  constexpr int BH = BN / 2, kSB = kTile + BH * kRowBytes, kSt = kPairRing / kSB, kLd = BN + 4;
  static_assert(128 * kLd * 4 <= kPairRing, "the sums fit over the ring");
  constexpr uint32_t kId = tc::idesc(F8, false, 256, BN);
  constexpr int kElems = F8 ? 128 : 64;
  constexpr uint32_t kTx = 2u * kSB;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kSt], empty[kSt], done;
  __shared__ uint32_t tmem_base;
  __shared__ int issued, consumed, failed;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = blockIdx.x % (2 * split), half = rank & 1u, lead = rank & ~1u;
  const int part = rank >> 1, tile = blockIdx.x / (2 * split), mt = (e.M + 255) / 256;
  const int m0 = tile % mt * 256 + (int)half * 128, n0 = tile / mt * BN;
  const int k_lo = (int)((long long)KB * part / split), k_hi = (int)((long long)KB * (part + 1) / split);
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (tid == 0) {
    for (int s = 0; s < kSt; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    issued = consumed = failed = 0;
    fence_mbar_init();
    tc::prefetch_map(&tmX);
    tc::prefetch_map(&tmW);
  }
  if (warp == 0) tc::alloc<2>(&tmem_base, 256);
  tc::fence_before();
  tc::cluster_sync();
  tc::fence_after();
  const uint32_t tmem = tmem_base;
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      int g = 0;
      for (int kb = k_lo; kb < k_hi; ++kb, ++g) {
        const int s = g % kSt, use = g / kSt;
        if (use > 0 && !mbar_wait_bounded(&empty[s], (uint32_t)((use - 1) & 1))) {
          failed = 1;
          break;
        }
        uint8_t* a = smem + s * kSB;
        if (half == 0) mbar_arrive_expect_tx(&full[s], kTx);
        const uint32_t fb = tc::cluster_addr(&full[s], lead);
        tc::tma_load_pair(a, &tmX, kb * kElems, m0, fb);
        tc::tma_load_pair(a + kTile, &tmW, kb * kElems, n0 + (int)half * BH, fb);
      }
      issued = g;
    }
  } else if (warp == 1) {
    if (lane == 0 && half == 0) {
      int g = 0;
      for (int kb = k_lo; kb < k_hi; ++kb, ++g) {
        const int s = g % kSt;
        if (!mbar_wait_bounded(&full[s], (uint32_t)((g / kSt) & 1))) {
          failed = 1;
          break;
        }
        tc::fence_after();
        const uint32_t a = smem_addr(smem + s * kSB), w = a + kTile;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          tc::mma<2, F8>(tmem, tc::desc_sw128(a + 32 * q, 16, 1024), tc::desc_sw128(w + 32 * q, 16, 1024), kId,
                         (g | q) != 0);
        tc::commit<2>(tc::cluster_addr(&empty[s], lead));
        tc::commit<2>(tc::cluster_addr(&empty[s], lead + 1));
      }
      consumed = g;
      tc::commit<2>(tc::cluster_addr(&done, lead));
      tc::commit<2>(tc::cluster_addr(&done, lead + 1));
    }
  }
  __syncwarp();
  if (!mbar_wait_bounded(&done, 0, e.tries)) failed = 1;
  tc::fence_after();
  __syncthreads();
  if (tid == 0 && failed) {  // a wait ran out: copies and products on their way end first
    atomicOr(flags, SV_FLAG_TIMEOUT);
    if (half == 0)
      for (int g = consumed; g < issued; ++g) (void)mbar_wait_bounded(&full[g % kSt], (uint32_t)((g / kSt) & 1), 64);
    (void)mbar_wait_bounded(&done, 0);
    for (uint32_t r = 0; r < 2u * split; ++r)  // (a half of the tile may be missing: all of it is NaN)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(tc::cluster_addr(&failed, r)), "r"(1) : "memory");
  }
  tc::cluster_sync();  // (both halves' copies have landed: the ring may be written)
  tc::fence_after();
  const bool lost = failed != 0;  // (the same in the whole cluster)
  float* sums = reinterpret_cast<float*>(smem);  // [128][kLd]
  if (warp >= 2) {
    const int lg = warp & 3, ch = (warp - 2) >> 2;
    float* row = sums + (lg * 32 + lane) * kLd;
#pragma unroll 1
    for (int k = ch * BH; k < (ch + 1) * BH; k += 16) {
      uint32_t v[16];
      tc::ld16(tmem + ((uint32_t)(lg * 32) << 16) + k, v);
      tc::ld_wait(v);
#pragma unroll
      for (int q = 0; q < 16; ++q) v[q] = lost ? kNan : v[q];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4*>(row + k + 4 * q) = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    }
  }
  tc::fence_before();
  tc::cluster_sync();
  const int rows = 128 / split, r0 = part * rows;
  const uint32_t base = smem_addr(sums);
  const int c = (tid % (BN / 4)) * 4, n = n0 + c;  // four columns of a thread
  constexpr int kLanes = kPairThreads / (BN / 4);   // rows at a time
  float sw[4], bias[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sw[j] = e.sw && n + j < e.N ? e.sw[n + j] : 1.f;
    bias[j] = e.bias && n + j < e.N ? bf16(e.bias + n + j) : 0.f;
  }
  const bool whole = e.vec && n + 4 <= e.N;
#pragma unroll 2
  for (int r = tid / (BN / 4); r < rows; r += kLanes) {
    const long long m = m0 + r0 + r;
    if (m >= e.M || n >= e.N) break;
    float res[4] = {0.f, 0.f, 0.f, 0.f};
    if (e.res) {
      if (e.out_f32) {
        const float* p = static_cast<const float*>(e.res) + m * e.ldr + n;
        if (whole) {
          const float4 a = *reinterpret_cast<const float4*>(p);
          res[0] = a.x, res[1] = a.y, res[2] = a.z, res[3] = a.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j < e.N) res[j] = p[j];
        }
      } else {
        const uint16_t* p = static_cast<const uint16_t*>(e.res) + m * e.ldr + n;
        if (whole) {
          const uint2 a = *reinterpret_cast<const uint2*>(p);
          res[0] = bf16_lo(a.x), res[1] = bf16_hi(a.x), res[2] = bf16_lo(a.y), res[3] = bf16_hi(a.y);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j < e.N) res[j] = bf16(p + j);
        }
      }
    }
    float of[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int j = 0; j < 4; ++j) of[q][j] = 0.f;
      if (q < split) {
        uint32_t at;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(at)
                     : "r"(base + 4u * ((r0 + r) * kLd + c)), "r"(2 * q + (int)half));
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(of[q][0]), "=f"(of[q][1]), "=f"(of[q][2]), "=f"(of[q][3])
                     : "r"(at)
                     : "memory");
      }
    }
    const float sx = e.sx ? e.sx[m] : 1.f;
    float z[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      z[j] = __fmaf_rn(((of[0][j] + of[1][j]) + of[2][j]) + of[3][j], sx * sw[j], bias[j]);
    activate(z, e.act);
    if (e.res) {
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] += res[j];
    }
    if (e.out_f32) {
      float* o = static_cast<float*>(e.out) + m * e.ldo + n;
      if (whole) {
        *reinterpret_cast<float4*>(o) = make_float4(z[0], z[1], z[2], z[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < e.N) o[j] = z[j];
      }
    } else {
      uint16_t* o = static_cast<uint16_t*>(e.out) + m * e.ldo + n;
      if (whole) {
        *reinterpret_cast<uint2*>(o) = make_uint2(tc::pack_bf16x2(z[0], z[1]), tc::pack_bf16x2(z[2], z[3]));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < e.N) o[j] = __bfloat16_as_ushort(__float2bfloat16_rn(z[j]));
      }
    }
  }
  tc::cluster_sync();  // no CTA leaves while another reads its sums
  tc::fence_after();
  if (warp == 0) tc::dealloc<2>(tmem, 256);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct Job {
  const LinearLaunch* L;
  Epilogue e;
  int KB;
  tc::EncodeTiledFn enc;
  cudaStream_t st;
};

static void config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, long long grid, int threads, int cluster,
                   int smem, cudaStream_t st) {
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3((unsigned)grid, 1, 1);
  cfg->blockDim = dim3((unsigned)threads, 1, 1);
  cfg->dynamicSmemBytes = (size_t)smem;
  cfg->stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = cluster > 1 ? 2 : 1;
}

// x's map (boxes of x_rows rows) and W's (w_rows)
static bool maps(const Job& j, bool f8, int x_rows, int w_rows, CUtensorMap* x, CUtensorMap* w, std::string* err) {
  const LinearLaunch& L = *j.L;
  const uint64_t es = f8 ? 1 : 2;
  return tc::make_map(j.enc, x, f8, L.x, (uint64_t)L.K, (uint64_t)L.M, (uint64_t)L.ldx * es, (uint32_t)x_rows, err) &&
         tc::make_map(j.enc, w, f8, L.W, (uint64_t)L.K, (uint64_t)L.N, (uint64_t)L.ldw * es, (uint32_t)w_rows, err);
}

// Sets the kernel's shared-memory limit, once per device.
template <typename K>
static bool prepared(K kernel, int smem, std::atomic<int>* cache, std::string* err) {
  const int d = current_device();
  if (d < 0) {
    *err = "no current device (or its ordinal is too high)";
    return false;
  }
  if (cache[d].load(std::memory_order_acquire)) return true;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) {
    *err = std::string("linear attributes: ") + cudaGetErrorString(e);
    return false;
  }
  cache[d].store(1, std::memory_order_release);
  return true;
}

static int launched(cudaError_t e, std::string* err) {
  if (e == cudaSuccess) return SV_OK;
  *err = std::string("linear launch: ") + cudaGetErrorString(e);
  return SV_ERR_CUDA;
}

template <int TM, bool F8>
static int launch_rows(const Job& j, std::string* err) {
  static std::atomic<int> cache[kMaxDevices];
  using S = RowsShape<TM>;
  auto k = rows_kernel<TM, F8>;
  if (!prepared(k, S::kSmem, cache, err)) return SV_ERR_CUDA;
  CUtensorMap x, w;
  if (!maps(j, F8, TM, 128, &x, &w, err)) return SV_ERR_CUDA;
  const long long tiles = (j.e.N + 127LL) / 128;
  int split = 1;
  while (split < 8 && ((tiles * split * 2 <= 2 * tc::num_sms() && j.KB >= 8 * split) || (j.e.out_f32 && j.KB > kChunk * split)))
    split *= 2;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  config(&cfg, attr, tiles * split, kRowsThreads, split, S::kSmem, j.st);
  return launched(cudaLaunchKernelEx(&cfg, k, x, w, j.e, j.KB, split, j.L->flags), err);
}

template <int BN, int MS, bool F8, bool LONG = false>
static int launch_pair(const Job& j, std::string* err) {
  static std::atomic<int> cache[kMaxDevices];
  auto k = pair_kernel<BN, MS, F8, LONG>;
  if (!prepared(k, kPairSmem, cache, err)) return SV_ERR_CUDA;
  CUtensorMap x, w;
  if (!maps(j, F8, 128, BN / 2, &x, &w, err)) return SV_ERR_CUDA;
  const long long tiles = ((j.e.M + MS * 256LL - 1) / (MS * 256)) * ((j.e.N + BN - 1LL) / BN);
  const long long pairs = tc::num_sms() / 2;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  config(&cfg, attr, 2 * (tiles < pairs ? tiles : pairs), kPairThreads, 2, kPairSmem, j.st);
  return launched(cudaLaunchKernelEx(&cfg, k, x, w, j.e, j.KB, j.L->flags), err);
}

// Clusters of 2 * split CTAs that fit the card at once (15 of 8, 36 of 4 measured).
template <int BN, bool F8>
static int split_clusters(int split) {
  static std::atomic<int> cache[2][kMaxDevices];  // clusters + 1
  const int d = current_device();
  if (d < 0) return 0;
  std::atomic<int>& slot = cache[split == 4][d];
  int n = slot.load(std::memory_order_acquire) - 1;
  if (n < 0) {
    auto k = split_kernel<BN, F8>;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    config(&cfg, attr, 2 * split, kPairThreads, 2 * split, kPairRing + 1024, nullptr);
    n = 0;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairRing + 1024) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess)
      n = 0;
    slot.store(n + 1, std::memory_order_release);
  }
  return n;
}

template <int BN, bool F8>
static int launch_split(const Job& j, int split, std::string* err) {
  static std::atomic<int> cache[kMaxDevices];
  auto k = split_kernel<BN, F8>;
  if (!prepared(k, kPairRing + 1024, cache, err)) return SV_ERR_CUDA;
  CUtensorMap x, w;
  if (!maps(j, F8, 128, BN / 2, &x, &w, err)) return SV_ERR_CUDA;
  const long long tiles = ((j.e.M + 255LL) / 256) * ((j.e.N + BN - 1LL) / BN);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  config(&cfg, attr, 2 * split * tiles, kPairThreads, 2 * split, kPairRing + 1024, j.st);
  return launched(cudaLaunchKernelEx(&cfg, k, x, w, j.e, j.KB, split, j.L->flags), err);
}

template <bool F8>
static int dispatch(const Job& j, std::string* err) {
  const int M = j.e.M, N = j.e.N;
  const long long pairs = tc::num_sms() / 2;
  if (!j.e.out_f32 || j.KB <= 8 * kChunk) {
    if (M <= 16) return launch_rows<16, F8>(j, err);
    if (M <= 32) return launch_rows<32, F8>(j, err);
    if (M <= 64) return launch_rows<64, F8>(j, err);
    if (M <= 128) return launch_rows<128, F8>(j, err);
  }
  // fewer tiles than half of the pairs, and K long enough to be worth the exchange
  const long long t256 = ((M + 255LL) / 256) * ((N + 255LL) / 256), t128 = ((M + 255LL) / 256) * ((N + 127LL) / 128);
  for (int split = 4; split >= 2; split /= 2) {
    if (j.KB < 8 * split || (j.e.out_f32 && j.KB > kChunk * split)) continue;
    if (t128 <= split_clusters<128, F8>(split)) return launch_split<128, F8>(j, split, err);
    if (t256 <= split_clusters<256, F8>(split)) return launch_split<256, F8>(j, split, err);
  }
  // Rows (ms x 256) and columns of a tile, by the clocks that they would take (all
  // measured).  A k block costs the MMAs' 2 ms BN, but no less than a slot's turn
  // through the ring (3650 over the slots: 0.32 us a block for 256 x 128 and for
  // 256 x 256 tiles in 6 slots), and a part more under full load (18% with one
  // sub-tile, which asks more of L2, and 12% with two).  An epilogue costs 37 a column
  // and sub-tile, 25 more with a residual, up to 15 more for the activation; behind the
  // last tile with one sub-tile, behind every one with two, which fill tensor memory.
  // 8192 x 4096 x 4096 bf16: 182 and 174 us (ms 1 and 2), with a residual 189 and 199;
  // K = 1024: 56 and 70.
  const int widths[4] = {256, 224, 192, 128};
  const int act_clocks[5] = {0, 0, 5, 15, 11};
  const int column = 37 + (j.e.res ? 25 : 0) + act_clocks[j.e.act];
  int bw = 256, bms = 1;
  long long best = -1;
  for (int ms = 1; ms <= 2; ++ms)
    for (int w : widths) {
      const long long tiles = ((M + ms * 256LL - 1) / (ms * 256)) * ((N + w - 1LL) / w);
      const long long rounds = (tiles + pairs - 1) / pairs, slots = kPairRing / (ms * kTile + w / 2 * kRowBytes);
      const long long block = (2 * ms * w > 3650 / slots ? 2 * ms * w : 3650 / slots) * (ms == 1 ? 118 : 112) / 100;
      const long long loop = block * j.KB, end = (long long)ms * w * column;
      const long long cost = ms == 1 ? rounds * (loop > end ? loop : end) + end : rounds * (loop + end);
      if (best < 0 || cost < best) {
        best = cost;
        bw = w;
        bms = ms;
      }
    }
  if (j.e.out_f32 && j.KB > kChunk) {
    const long long tiles = ((M + 255LL) / 256) * ((N + 255LL) / 256);
    return tiles >= pairs ? launch_pair<256, 1, F8, true>(j, err) : launch_pair<128, 1, F8, true>(j, err);
  }
  switch (bw * 2 + bms - 1) {
    case 256 * 2: return launch_pair<256, 1, F8>(j, err);
    case 256 * 2 + 1: return launch_pair<256, 2, F8>(j, err);
    case 224 * 2: return launch_pair<224, 1, F8>(j, err);
    case 224 * 2 + 1: return launch_pair<224, 2, F8>(j, err);
    case 192 * 2: return launch_pair<192, 1, F8>(j, err);
    case 192 * 2 + 1: return launch_pair<192, 2, F8>(j, err);
    case 128 * 2: return launch_pair<128, 1, F8>(j, err);
    default: return launch_pair<128, 2, F8>(j, err);
  }
}

}  // namespace lin

int linear_launch(const LinearLaunch& L, std::string* err) {
  lin::Job j;
  j.L = &L;
  j.enc = tc::encoder(err);
  if (!j.enc) return SV_ERR_CUDA;
  const int es = L.in_dtype == SV_BF16 ? 2 : 1, os = L.out_dtype == SV_BF16 ? 2 : 4;
  const bool vec = reinterpret_cast<uintptr_t>(L.out) % 16 == 0 && L.ldo * os % 16 == 0 &&
                   (!L.residual || (reinterpret_cast<uintptr_t>(L.residual) % 16 == 0 && L.ldr * os % 16 == 0));
  j.e = {L.x_scale, L.w_scale, static_cast<const uint16_t*>(L.bias), L.residual, L.ldr, L.out, L.ldo,
         L.act, L.out_dtype == SV_F32 ? 1 : 0, L.M, L.N, vec ? 1 : 0, (uint32_t)L.wait_tries};
  j.KB = (int)(((long long)L.K * es + lin::kRowBytes - 1) / lin::kRowBytes);
  j.st = static_cast<cudaStream_t>(L.stream);
  return L.in_dtype == SV_BF16 ? lin::dispatch<false>(j, err) : lin::dispatch<true>(j, err);
}

}  // namespace sv
