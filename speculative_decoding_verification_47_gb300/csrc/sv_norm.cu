// Residual addition, RMSNorm and 8-bit quantisation of a row in one pass: the
// norm of "Self-speculative decoding with layer skip and KV reuse" §3.1
// between two layers.
//
//   s = x + residual,  y = w s / sqrt(mean(s^2) + eps)
//   e4m3:  c = max(max|y| / 448, 2^-126),  q = rn(y / c)
//
// max|y| = rsqrt(..) * max|w s|, so the sum of squares and the maximum come
// from the same pass and one reduction.  The row stays in registers (float32)
// between that pass and the scaling: x and residual are read once.  s is
// rounded only where it is stored; y comes from the unrounded sum.
//
// Bound by memory.  A CTA (or a warp) per row, all of its loads before the first sum; long rows,
// more of them than fit the card at once: CTAs that stay, with the next rows on their way into
// shared memory by bulk copies while one is reduced and stored.  Measured with inputs outside of
// L2: 16384 x 8192 float32 to bf16 264 us (7.1 TB/s), bf16 with a residual to e4m3 162 us
// (5.8 TB/s), 2304 x 4096 13.0 us (four rows a CTA: the first copies and the rows' chains of
// reduction and stores, 63% of the issue slots), one row 1.8 us (latencies).
#include <atomic>
#include <cstdint>

#include "sv_common.cuh"
#include "sv_internal.h"

namespace sv {
namespace norm {

constexpr float kE4M3Max = 448.f;
constexpr float kTiny = 1.17549435e-38f;  // 2^-126: 1 / c stays finite

constexpr int kShifted = -8;  // in place of a vector's width: runs of 8 at a common phase

struct Args {
  const void* x;
  long long ldx;
  const void* res;
  long long ldr;
  const uint16_t* w;
  float eps;
  void* sum;
  long long lds;
  void* out;
  long long ldo;
  float* scale;
  int M, H;
  uint32_t tries;  // of a wait for a row's copy
};

// max that keeps a NaN (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Vectors of VEC elements as 32-bit words (bf16: two to a word, e4m3: four), so that
// widening is a shift or a mask and narrowing one instruction for two values.
template <int N>
struct alignas(N * 4 > 16 ? 16 : N * 4) Words {
  uint32_t v[N];
};

template <int VEC>
__device__ __forceinline__ void load(const uint16_t* p, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = __uint_as_float((uint32_t)*p << 16);
  } else {
    const Words<VEC / 2> h = *reinterpret_cast<const Words<VEC / 2>*>(p);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      f[2 * i] = bf16_lo(h.v[i]);
      f[2 * i + 1] = bf16_hi(h.v[i]);
    }
  }
}
template <int VEC>
__device__ __forceinline__ void load(const float* p, float (&f)[VEC]) {
  const Words<VEC> h = *reinterpret_cast<const Words<VEC>*>(p);
#pragma unroll
  for (int i = 0; i < VEC; ++i) f[i] = __uint_as_float(h.v[i]);
}
template <int VEC>
__device__ __forceinline__ void store(uint16_t* p, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    *p = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
  } else {
    Words<VEC / 2> h;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const __nv_bfloat162 two = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      h.v[i] = *reinterpret_cast<const uint32_t*>(&two);
    }
    *reinterpret_cast<Words<VEC / 2>*>(p) = h;
  }
}
template <int VEC>
__device__ __forceinline__ void store(float* p, const float (&f)[VEC]) {
  Words<VEC> h;
#pragma unroll
  for (int i = 0; i < VEC; ++i) h.v[i] = __float_as_uint(f[i]);
  *reinterpret_cast<Words<VEC>*>(p) = h;
}

// two values to e4m3 (round to nearest, out of range to +-448, NaN kept)
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int VEC>
__device__ __forceinline__ void store8(uint8_t* p, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    *p = (uint8_t)e4m3x2(f[0], 0.f);
  } else if constexpr (VEC == 2) {
    *reinterpret_cast<uint16_t*>(p) = e4m3x2(f[0], f[1]);
  } else {
    Words<VEC / 4> h;
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      h.v[i] = (uint32_t)e4m3x2(f[4 * i], f[4 * i + 1]) | ((uint32_t)e4m3x2(f[4 * i + 2], f[4 * i + 3]) << 16);
    *reinterpret_cast<Words<VEC / 4>*>(p) = h;
  }
}

// Sum and maximum over the threads of a row, to all of them (one barrier: calls in a
// row need places of their own).
__device__ __forceinline__ void reduce(float (&part)[2][32], float& sum, float& top) {
  const int t = threadIdx.x, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (warps == 1) return;  // (else blockDim.y is 1)
  if ((t & 31) == 0) {
    part[0][t >> 5] = sum;
    part[1][t >> 5] = top;
  }
  __syncthreads();
  sum = (t & 31) < warps ? part[0][t & 31] : 0.f;
  top = (t & 31) < warps ? part[1][t & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
}

// y / c for all values of a row by its scale's reciprocal in two words: off by little more than
// half a step, as a division is.  (With one word 73 of 155584 quotients of bf16 values went to
// the other side of a border between two e4m3 values.)
struct Divisor {
  float hi, lo;
  __device__ __forceinline__ explicit Divisor(float c) : hi(1.f / c) {
    lo = c < INFINITY ? __fmaf_rn(-hi, c, 1.f) * hi : 0.f;
  }
};

// y = v r w, divided for an 8-bit result, then two values an instruction.
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <bool Q8, int VEC>
__device__ __forceinline__ void results(const float (&v)[VEC], float r, const float (&w)[VEC], const Divisor& by,
                                        float (&y)[VEC]) {
  if constexpr (VEC == 1 || !Q8) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      y[i] = v[i] * r * w[i];
      if (Q8) y[i] = __fmaf_rn(y[i], by.hi, y[i] * by.lo);
    }
  } else {
    const F2 r2 = f2_pack(r, r), hi = f2_pack(by.hi, by.hi), lo = f2_pack(by.lo, by.lo);
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
      F2 t = f2_mul(f2_mul(f2_pack(v[i], v[i + 1]), r2), f2_pack(w[i], w[i + 1]));
      t = f2_fma(t, hi, f2_mul(t, lo));
      f2_unpack(t, y[i], y[i + 1]);
    }
  }
}

// A mean of squares (and eps) whose squares left float32's range: values above 1.8e19, or
// below 1e-18 with so small an eps.
__device__ __forceinline__ bool far(float mean) { return mean < 0x1p-120f || mean == INFINITY; }

// Such a row, by the threads that have it and from memory again: it is scaled by a power of
// two p that brings the larger of its largest magnitude and sqrt(eps) next to 1, and
//   y = w (p s) / sqrt(mean((p s)^2) + p^2 eps).
// p is 1 where no scaling helps (a value that is not finite, nothing but zeros).  From
// memory, so that the usual path's registers are not held for it.
template <typename T, bool Q8>
__device__ __forceinline__ void far_row(const Args& a, long long m, float (&part)[2][32]) {
  const int t = threadIdx.x, n = blockDim.x;
  const T* x = static_cast<const T*>(a.x) + m * a.ldx;
  const T* res = a.res ? static_cast<const T*>(a.res) + m * a.ldr : nullptr;
  float s[1], r[1], w[1], y[1], none = 0.f, big = 0.f, p = 1.f, ss = 0.f, top = 0.f, c = 1.f;
  auto sum_at = [&](long long k) {
    load<1>(x + k, s);
    if (res) {
      load<1>(res + k, r);
      s[0] += r[0];
    }
    return s[0];
  };
  auto all = [&](float& sum, float& most) {
    if (n > 32)
      __syncthreads();  // (part[] is free, and what the row's other threads stored lies before it)
    else
      __syncwarp();
    reduce(part, sum, most);
  };
#pragma unroll 1
  for (long long k = t; k < a.H; k += n) big = max_nan(big, fabsf(sum_at(k)));
  all(none, big);
  const float ref = fmaxf(big, sqrtf(a.eps));
  if (big < INFINITY && ref < INFINITY && ref > 0.f) {
    const int e = (int)(__float_as_uint(ref) >> 23) - 127;
    p = __uint_as_float((uint32_t)(127 - min(max(e, -126), 126)) << 23);
  }
#pragma unroll 1
  for (long long k = t; k < a.H; k += n) {
    const float v = sum_at(k) * p;
    ss = __fmaf_rn(v, v, ss);
  }
  all(ss, none);
  const float inv = rsqrtf(ss / (float)a.H + a.eps * p * p);
  if (Q8) {
#pragma unroll 1
    for (long long k = t; k < a.H; k += n) {
      load<1>(a.w + k, w);
      top = max_nan(top, fabsf(sum_at(k) * p * inv * w[0]));
    }
    all(none, top);
    c = top / kE4M3Max;
    if (c < kTiny) c = kTiny;  // (a NaN stays)
    if (t == 0) a.scale[m] = c;
  }
#pragma unroll 1
  for (long long k = t; k < a.H; k += n) {
    load<1>(a.w + k, w);
    y[0] = sum_at(k) * p * inv * w[0] / c;
    if (a.sum) store<1>(static_cast<T*>(a.sum) + m * a.lds + k, s);
    if (Q8)
      store8<1>(static_cast<uint8_t*>(a.out) + m * a.ldo + k, y);
    else
      store<1>(static_cast<uint16_t*>(a.out) + m * a.ldo + k, y);
  }
}

// One row per blockDim.x threads (blockDim.y rows per CTA only with one warp
// per row).  Thread t holds elements (j * blockDim.x + t) * VEC .., j < NV;
// rows longer than NV * VEC * blockDim.x are read again for the scaling, each
// element by the thread that overwrites it.
//
// SHIFT: rows that start anywhere, all arrays' at the same place of an aligned run of
// VEC elements (`phase`).  The vectors are the aligned runs, so the first and the last
// one of a row may be cut: these go element by element, as zeros outside of the row.
template <typename T, bool Q8, int VEC, int NV, bool SHIFT = false>
__global__ void __launch_bounds__(1024) norm_kernel(const Args a) {
  __shared__ float part[2][32];
  pdl_launch_dependents();
  const int t = threadIdx.x, n = blockDim.x;
  const long long m = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = m < a.M;
  const T* x = static_cast<const T*>(a.x) + (live ? m : 0) * a.ldx;
  const T* res = a.res ? static_cast<const T*>(a.res) + (live ? m : 0) * a.ldr : nullptr;
  const int phase = SHIFT && live ? (int)((m * a.ldx) & (VEC - 1)) : 0;
  pdl_wait();  // the launch may overlap the kernel that wrote x

  auto whole = [&](int k) { return !SHIFT || (k >= 0 && k + VEC <= a.H); };
  auto get = [&](const auto* from, int k, float (&f)[VEC]) {
    if (whole(k)) {
      load<VEC>(from + k, f);
      return;
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float one[1] = {0.f};
      if (k + i >= 0 && k + i < a.H) load<1>(from + k + i, one);
      f[i] = one[0];
    }
  };
  // the weight's run from k on as words of two (one element: alone), and widened
  constexpr int WW = VEC > 1 ? VEC / 2 : 1;
  auto weight_words = [&](int k, uint32_t (&h)[WW]) {
    if constexpr (VEC == 1) {
      h[0] = a.w[k];
    } else if constexpr (!SHIFT) {
      const Words<WW> in = *reinterpret_cast<const Words<WW>*>(a.w + k);
#pragma unroll
      for (int i = 0; i < WW; ++i) h[i] = in.v[i];
    } else if (whole(k)) {  // (words on 4 bytes, the elements between them)
      const uint32_t* at = reinterpret_cast<const uint32_t*>(a.w + (k & ~1));
#pragma unroll
      for (int i = 0; i < WW; ++i) h[i] = at[i];
      if (k & 1) {
        const uint32_t last = a.w[k + VEC - 1];
#pragma unroll
        for (int i = 0; i < WW; ++i) h[i] = __funnelshift_r(h[i], i + 1 < WW ? h[i + 1] : last, 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const uint32_t one = k + i >= 0 && k + i < a.H ? a.w[k + i] : 0u;
        h[i / 2] = i & 1 ? h[i / 2] | one << 16 : one;
      }
    }
  };
  auto widen = [&](const uint32_t (&h)[WW], float (&f)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = i & 1 ? bf16_hi(h[i / 2]) : bf16_lo(h[i / 2]);
  };
  auto weight = [&](int k, float (&f)[VEC]) {
    uint32_t h[WW];
    weight_words(k, h);
    widen(h, f);
  };
  auto sum_at = [&](int k, float (&s)[VEC]) {
    get(x, k, s);
    if (res) {
      float r[VEC];
      get(res, k, r);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[i] += r[i];
    }
  };
  float s[NV][VEC], ss = 0.f, top = 0.f;
  uint32_t held[VEC == 1 ? 1 : NV][WW];
  if constexpr (VEC > 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (j * n + t) * VEC - phase;
      if (k < a.H) weight_words(k, held[j]);
    }
  }
  auto gather = [&](const float (&v)[VEC], const float (&w)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      ss = __fmaf_rn(v[i], v[i], ss);
      if (Q8) top = max_nan(top, fabsf(v[i] * w[i]));
    }
  };
  if constexpr (!SHIFT && VEC * sizeof(T) >= 4) {
    // every load before the first sum waits for one
    using Raw = Words<VEC * sizeof(T) / 4>;
    Raw rx[NV], rr[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (j * n + t) * VEC;
#pragma unroll
      for (int i = 0; i < (int)(sizeof(Raw) / 4); ++i) rx[j].v[i] = rr[j].v[i] = 0;
      if (k < a.H) rx[j] = *reinterpret_cast<const Raw*>(x + k);
    }
    if (res) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int k = (j * n + t) * VEC;
        if (k < a.H) rr[j] = *reinterpret_cast<const Raw*>(res + k);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        if constexpr (sizeof(T) == 4)
          s[j][i] = __uint_as_float(rx[j].v[i]) + (res ? __uint_as_float(rr[j].v[i]) : 0.f);
        else
          s[j][i] = (i & 1 ? bf16_hi(rx[j].v[i / 2]) : bf16_lo(rx[j].v[i / 2])) +
                    (res ? (i & 1 ? bf16_hi(rr[j].v[i / 2]) : bf16_lo(rr[j].v[i / 2])) : 0.f);
      }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (j * n + t) * VEC - phase;
      if (k < a.H) {
        sum_at(k, s[j]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[j][i] = 0.f;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int k = (j * n + t) * VEC - phase;
    if (k < a.H) {
      float w[VEC];
      if constexpr (VEC > 1)
        widen(held[j], w);
      else
        weight(k, w);
      gather(s[j], w);
    }
  }
  for (long long k = (long long)(NV * n + t) * VEC; k < a.H; k += (long long)n * VEC) {
    float v[VEC];
    sum_at((int)k, v);
    float w[VEC];
    weight((int)k, w);
    gather(v, w);
  }
  reduce(part, ss, top);
  const float mean = ss / (float)a.H + a.eps;
  float r = rsqrtf(mean);
  // |w s| may leave float32's range where |w s r| does not (s far from 1 and w
  // with it): then the maximum is taken again, from the values themselves
  if (Q8 && !(top > 1e-30f && top < 1e30f)) {  // (the same in every thread of the row)
    top = 0.f;
    auto again = [&](const float (&v)[VEC], int k) {
      float w[VEC];
      weight(k, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) top = max_nan(top, fabsf(v[i] * r * w[i]));
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (j * n + t) * VEC - phase;
      if (k < a.H) again(s[j], k);
    }
    for (long long k = (long long)(NV * n + t) * VEC; k < a.H; k += (long long)n * VEC) {
      float v[VEC];
      sum_at((int)k, v);
      again(v, (int)k);
    }
    if (n > 32) __syncthreads();  // (part[] is free again)
    float none = 0.f;
    reduce(part, none, top);
  } else {
    top *= r;
  }
  if (!live) return;
  float c = top / kE4M3Max;
  if (c < kTiny) c = kTiny;  // (a NaN stays)
  if (Q8 && t == 0) a.scale[m] = c;
  const Divisor by(c);
  // (a row that is done again below: its sum may lie over x, which that reads)
  T* sum = a.sum && !far(mean) ? static_cast<T*>(a.sum) + m * a.lds : nullptr;
  auto finish = [&](const float (&v)[VEC], const float (&w)[VEC], int k) {
    float y[VEC];
    results<Q8>(v, r, w, by, y);
    if (whole(k)) {
      if (sum) store<VEC>(sum + k, v);
      if (Q8)
        store8<VEC>(static_cast<uint8_t*>(a.out) + m * a.ldo + k, y);
      else
        store<VEC>(static_cast<uint16_t*>(a.out) + m * a.ldo + k, y);
      return;
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      if (k + i < 0 || k + i >= a.H) continue;
      const float v1[1] = {v[i]}, y1[1] = {y[i]};
      if (sum) store<1>(sum + k + i, v1);
      if (Q8)
        store8<1>(static_cast<uint8_t*>(a.out) + m * a.ldo + k + i, y1);
      else
        store<1>(static_cast<uint16_t*>(a.out) + m * a.ldo + k + i, y1);
    }
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int k = (j * n + t) * VEC - phase;
    if (k < a.H) {
      float w[VEC];
      if constexpr (VEC > 1)
        widen(held[j], w);
      else
        weight(k, w);
      finish(s[j], w, k);
    }
  }
  for (long long k = (long long)(NV * n + t) * VEC; k < a.H; k += (long long)n * VEC) {
    float v[VEC], w[VEC];
    sum_at((int)k, v);
    weight((int)k, w);
    finish(v, w, (int)k);
  }
  if (far(mean)) far_row<T, Q8>(a, m, part);  // (the same in every thread of the row)
}

// ---------------------------------------------------------------------------
// Rows of 16-byte words through a ring of shared memory: `slots` rows of x and
// residual ahead.  Thread t holds elements (j * blockDim.x + t) * 8 .., j < 2.
// 2304 x 12288 bf16 with a residual to e4m3: 32 us, 46 with a CTA per row, whose loads,
// reduction and stores follow one another.
// ---------------------------------------------------------------------------
constexpr int kRing = 8;  // slots at most

__device__ __forceinline__ void bulk(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

template <typename T, bool Q8>
__global__ void __launch_bounds__(1024, 1) ring_kernel(const Args a, int slots) {
  constexpr int VEC = 8, NV = 2;
  extern __shared__ __align__(16) uint8_t ring[];  // the slots
  __shared__ float part[4][2][32];
  __shared__ __align__(8) uint64_t full[kRing];
  const int t = threadIdx.x, n = blockDim.x;
  const uint32_t row_bytes = (uint32_t)a.H * sizeof(T), slot_bytes = a.res ? 2 * row_bytes : row_bytes;
  pdl_launch_dependents();
  if (t == 0) {
    for (int s = 0; s < slots; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  pdl_wait();  // the launch may overlap the kernel that wrote x
  __syncthreads();
  auto ask = [&](long long m, int s) {  // (one thread)
    mbar_arrive_expect_tx(&full[s], slot_bytes);
    bulk(ring + s * slot_bytes, static_cast<const T*>(a.x) + m * a.ldx, row_bytes, &full[s]);
    if (a.res) bulk(ring + s * slot_bytes + row_bytes, static_cast<const T*>(a.res) + m * a.ldr, row_bytes, &full[s]);
  };
  if (t == 0)
    for (int s = 0; s < slots && blockIdx.x + (long long)s * gridDim.x < a.M; ++s)
      ask(blockIdx.x + (long long)s * gridDim.x, s);
  Words<VEC / 2> w[NV];  // a thread's columns are the same in every row
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int k = (j * n + t) * VEC;
    if (k < a.H) w[j] = *reinterpret_cast<const Words<VEC / 2>*>(a.w + k);
  }
  auto weight = [&](int j, float (&f)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = i & 1 ? bf16_hi(w[j].v[i / 2]) : bf16_lo(w[j].v[i / 2]);
  };
  int slot = 0, turn = 0, late = 0x7fffffff;  // the turn whose copy did not come in time
  uint32_t phase = 0;
  for (long long m = blockIdx.x; m < a.M; m += gridDim.x, ++turn) {
    // A thread whose wait runs out waits no more, asks for no more and brings NaN into
    // this row and every one behind it.
    if (late > turn && !mbar_wait_bounded(&full[slot], phase, a.tries)) late = turn;
    const T* x = reinterpret_cast<const T*>(ring + slot * slot_bytes);
    float s[NV][VEC], ss = 0.f, top = 0.f;
    F2 squares = f2_pack(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (j * n + t) * VEC;
      if (k < a.H) {
        load<VEC>(x + k, s[j]);
        if (a.res) {
          float r[VEC];
          load<VEC>(x + a.H + k, r);
#pragma unroll
          for (int i = 0; i < VEC; ++i) s[j][i] += r[i];
        }
        float v[VEC];
        if (Q8) weight(j, v);
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
          const F2 two = f2_pack(s[j][i], s[j][i + 1]);
          squares = f2_fma(two, two, squares);
          if (Q8) {
            float p0, p1;
            f2_unpack(f2_mul(two, f2_pack(v[i], v[i + 1])), p0, p1);
            top = max_nan(top, max_nan(fabsf(p0), fabsf(p1)));
          }
        }
      }
    }
    float even, odd;
    f2_unpack(squares, even, odd);
    ss = even + odd;
    if (late <= turn) {
      ss = top = __int_as_float(0x7fffffff);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[j][i] = ss;
    }
    reduce(part[turn & 1], ss, top);  // (every thread has read the slot)
    if (t == 0 && late > turn && m + (long long)slots * gridDim.x < a.M) ask(m + (long long)slots * gridDim.x, slot);
    if (++slot == slots) {
      slot = 0;
      phase ^= 1;
    }
    const float mean = ss / (float)a.H + a.eps, r = rsqrtf(mean);
    if (Q8 && !(top > 1e-30f && top < 1e30f)) {  // as in norm_kernel
      top = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int k = (j * n + t) * VEC;
        if (k < a.H) {
          float v[VEC];
          weight(j, v);
#pragma unroll
          for (int i = 0; i < VEC; ++i) top = max_nan(top, fabsf(s[j][i] * r * v[i]));
        }
      }
      float none = 0.f;
      reduce(part[2 + (turn & 1)], none, top);
    } else {
      top *= r;
    }
    float c = top / kE4M3Max;
    if (c < kTiny) c = kTiny;  // (a NaN stays)
    if (Q8 && t == 0) a.scale[m] = c;
    const Divisor by(c);
    T* sum = a.sum && !far(mean) ? static_cast<T*>(a.sum) + m * a.lds : nullptr;  // (as in norm_kernel)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (j * n + t) * VEC;
      if (k < a.H) {
        float v[VEC], y[VEC];
        weight(j, v);
        results<Q8>(s[j], r, v, by, y);
        if (sum) store<VEC>(sum + k, s[j]);
        if (Q8)
          store8<VEC>(static_cast<uint8_t*>(a.out) + m * a.ldo + k, y);
        else
          store<VEC>(static_cast<uint16_t*>(a.out) + m * a.ldo + k, y);
      }
    }
    if (far(mean)) far_row<T, Q8>(a, m, part[2 + (turn & 1)]);
  }
  if (t == 0 && late < turn)  // (copies on their way end before the CTA does)
    for (int g = late; g < late + slots && blockIdx.x + (long long)g * gridDim.x < a.M; ++g)
      (void)mbar_wait_bounded(&full[g % slots], (uint32_t)((g / slots) & 1), 64);
}

// The ring's launch: CTAs of H / 16 threads, as many as an SM's threads and shared
// memory hold with `slots` rows each.  `ctas` = 0 if a row does not fit.
static void ring_shape(const Args& a, int es, int threads, int* slots, int* ctas, int* smem) {
  const int slot = a.H * es * (a.res ? 2 : 1), room = 200 * 1024;
  int per_sm = 1024 / threads;  // (64 registers a thread)
  if (per_sm > 8) per_sm = 8;
  *ctas = 0;
  for (; per_sm >= 1; --per_sm) {
    // (less 2 H: a third slot at H = 4096 and 8192 gains nothing, 16384 x 8192 168 us, 161 with two)
    const int fits = (room / per_sm - a.H * 2 - 2048) / slot;
    if (fits < 2) continue;
    *slots = fits < kRing ? fits : kRing;
    *smem = *slots * slot;
    *ctas = per_sm;
    return;
  }
}

template <typename T, bool Q8>
static cudaError_t launch_ring(const Args& a, int threads, int slots, int ctas, int smem, cudaStream_t st) {
  static std::atomic<int> ready[kMaxDevices];
  const int d = current_device();
  if (d < 0) return cudaErrorInvalidDevice;
  int sms = ready[d].load(std::memory_order_acquire);
  if (sms == 0) {
    cudaError_t e = cudaFuncSetAttribute(ring_kernel<T, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, 204 * 1024);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d);
    if (e != cudaSuccess) return e;
    ready[d].store(sms, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.M < sms * ctas ? a.M : sms * ctas), 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ring_kernel<T, Q8>, a, slots);
}

template <typename T, bool Q8, int VEC, int NV, bool SHIFT = false>
static cudaError_t launch(const Args& a, int threads, int rows, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.M + (long long)rows - 1) / rows), 1, 1);
  cfg.blockDim = dim3((unsigned)threads, (unsigned)rows, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_kernel<T, Q8, VEC, NV, SHIFT>, a);
}

template <typename T, bool Q8>
static cudaError_t dispatch(const Args& a, int vec, cudaStream_t st) {
  constexpr int kPer = 16;  // elements a thread keeps
  int threads = 32;  // (not only powers of two: 2048 x 4097 29.6 us with 512 threads, 25.3 with 288)
  const int spread = a.H + (vec == kShifted ? 7 : 0);
  while (threads < 1024 && (long long)threads * kPer < spread) threads += 32;
  const int rows = threads == 32 ? 4 : 1;
  // The ring: rows in whole 16-byte words, more of them than the card holds CTAs of the plain
  // kernel at once (1024 threads an SM), and long ones.  Inputs outside of L2, ring and plain,
  // us: with a residual to e4m3 2304 x 4096 13.0 and 14.1, 4096 x 6144 30 and 37, 2304 x 12288
  // 32 and 46, but 16384 x 2048 42 and 38, 5000 x 1024 11.3 and 8.3; to bf16 4096 x 6144 36 and
  // 37, 16384 x 4096 89 and 78; without a residual 16384 x 2048 28 and 30, 16384 x 8192 101 and
  // 130, 5000 x 1024 9.0 and 7.6.  Not for float32 rows: twice the bytes are in flight anyway,
  // and half as many rows fit the ring (16384 x 8192: 263 by the plain kernel, 317 by the ring).
  const int ring_from = a.res ? (Q8 ? 4096 : 4097) : 2048;
  if (sizeof(T) == 2 && vec == 8 && a.H >= ring_from && a.H <= kPer * threads && a.M > 152LL * (1024 / threads)) {
    int slots = 0, ctas = 0, smem = 0;
    ring_shape(a, sizeof(T), threads, &slots, &ctas, &smem);
    if (sizeof(T) == 2 && ctas > 0) return launch_ring<uint16_t, Q8>(a, threads, slots, ctas, smem, st);
  }
  if (vec == 8) return launch<T, Q8, 8, kPer / 8>(a, threads, rows, st);
  if (vec == kShifted && spread <= threads * kPer) return launch<T, Q8, 8, kPer / 8, true>(a, threads, rows, st);
  if (vec == 2) return launch<T, Q8, 2, kPer / 2>(a, threads, rows, st);
  return launch<T, Q8, 1, kPer>(a, threads, rows, st);
}

}  // namespace norm

int norm_launch(const NormLaunch& L, std::string* err) {
  norm::Args a = {L.x, L.ldx, L.residual, L.ldr, static_cast<const uint16_t*>(L.w), L.eps,
                  L.residual_out, L.ldro, L.out, L.ldo, L.out_scale, L.M, L.H, (uint32_t)L.wait_tries};
  const size_t es = L.dtype == SV_BF16 ? 2 : 4, os = L.out_dtype == SV_BF16 ? 2 : 1;
  // the widest vector that every row of every array starts on a multiple of
  auto fits = [&](int v) {
    auto on = [&](const void* p, long long ld, size_t e) {
      const size_t bytes = v * e > 16 ? 16 : v * e;
      return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (L.M == 1 || ld * e % bytes == 0);
    };
    return L.H % v == 0 && on(L.x, L.ldx, es) && (!L.residual || on(L.residual, L.ldr, es)) &&
           (!L.residual_out || on(L.residual_out, L.ldro, es)) && on(L.w, 0, 2) && on(L.out, L.ldo, os);
  };
  // Odd rows: runs of 8 at a phase that a row's arrays share.  2048 x 4097 bf16 to e4m3
  // 28.7 us element by element, 25.3 in runs; 1 x 5001 4.9 and 3.1; but 12000 x 33 (a
  // warp per row, most of its runs cut) 9.3 and 10.2.
  auto shares = [&](const void* p, long long ld, size_t e) {
    return reinterpret_cast<uintptr_t>(p) % (e == 1 ? 8 : 16) == 0 && (L.M == 1 || (ld - L.ldx) % 8 == 0);
  };
  const bool shifted = shares(L.x, L.ldx, es) && (!L.residual || shares(L.residual, L.ldr, es)) &&
                       (!L.residual_out || shares(L.residual_out, L.ldro, es)) && shares(L.out, L.ldo, os) &&
                       reinterpret_cast<uintptr_t>(L.w) % 4 == 0 && L.H > 512 && L.H + 7LL <= 16 * 1024;
  const int vec = fits(8) ? 8 : (fits(2) ? 2 : (shifted ? norm::kShifted : 1));
  cudaStream_t st = static_cast<cudaStream_t>(L.stream);
  const bool q8 = L.out_dtype == SV_E4M3;
  cudaError_t e;
  if (L.dtype == SV_BF16)
    e = q8 ? norm::dispatch<uint16_t, true>(a, vec, st) : norm::dispatch<uint16_t, false>(a, vec, st);
  else
    e = q8 ? norm::dispatch<float, true>(a, vec, st) : norm::dispatch<float, false>(a, vec, st);
  if (e != cudaSuccess) {
    *err = std::string("residual norm launch: ") + cudaGetErrorString(e);
    return SV_ERR_CUDA;
  }
  return SV_OK;
}

}  // namespace sv
