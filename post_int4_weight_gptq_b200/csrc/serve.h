// Shared pieces of the 8-bit serving entries (int8.cu, kv8.cu, kv8_attn.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace piq {

// Largest contraction whose int32 sum is exact for any codes: 128 * 128 * in < 2^31.
constexpr int64_t kInt8MaxIn = 131064;

// How one int8 product is cut into tiles (int8_gemm.cu).
struct Int8Plan {
  bool pair;   // tiles of 256 channels on two CTAs, else 128 on one
  int nt;      // tokens of a tile
  int slices;  // of k
};
Int8Plan plan_int8(int64_t tokens, int64_t out, int64_t in, int sms);
// Y = (qx W^T) sx sw + bias; qx, W int8 with 16-byte aligned rows, sx 16-byte aligned.
int launch_int8_gemm(const int8_t* qx, int64_t ldq, const float* sx, int64_t tokens, int64_t in,
                     const int8_t* W, int64_t out, int64_t ldw, const float* sw, const float* bias,
                     void* Y, int dtype, int64_t ldy, int32_t* status, cudaStream_t stream);

// cuTensorMapEncodeTiled of the loaded driver, nullptr if it has none.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder();

// The limit of the waits inside the kernels launched from now on
// (piq_serving_wait_limit).
uint64_t serving_wait_ns();

// A wait bounded by `limit` ns that reports to the caller's status words.  Who gives up
// makes the results that depend on the wait NaN, and no CTA ends with copies or products
// of its own under way: those are waited for with drain_bar.  Without mbar_wait's
// suspend hint, as these waits are short.
__device__ __forceinline__ void note_status(int32_t* status, int code, int detail);
__device__ __forceinline__ bool try_wait_now(uint64_t* bar, uint32_t parity) {  // may sleep
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool test_now(uint64_t* bar, uint32_t parity) {  // does not
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
constexpr uint64_t kBriefNs = 1000000;  // limits below it look at the clock every time
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, uint64_t limit,
                                         int32_t* status, int where) {
  if (try_wait_now(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  const int tries = limit < kBriefNs ? 1 : 64;
  for (;;) {
    for (int i = 0; i < tries; ++i)
      if (try_wait_now(bar, parity)) return true;
    if (global_timer_ns() - t0 >= limit) {
      note_status(status, PIQ_ERR_TIMEOUT, where);
      return false;
    }
  }
}
// The same for a whole warp, which goes on or gives up together.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint64_t limit,
                                          int32_t* status, int where) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, limit, status, where));
}
// For waits so short that one sleeping try outlasts them, whatever the limit: below
// kBriefNs without sleeping.
__device__ __forceinline__ bool wait_warp_short(uint64_t* bar, uint32_t parity, uint64_t limit,
                                                int32_t* status, int where) {
  bool ok = test_now(bar, parity);
  if (!ok) {
    if (limit >= kBriefNs) {
      ok = wait_bar(bar, parity, limit, status, where);
    } else {
      const uint64_t t0 = global_timer_ns();
      while (!(ok = test_now(bar, parity)) && global_timer_ns() - t0 < limit) {
      }
      if (!ok) note_status(status, PIQ_ERR_TIMEOUT, where);
    }
  }
  return __all_sync(0xffffffffu, ok);
}
// Waits, up to kWaitLimitNs from t0 on, for what is under way and will arrive on `bar`.
__device__ __forceinline__ void drain_bar(uint64_t* bar, uint32_t parity, uint64_t t0) {
  while (!try_wait_now(bar, parity) && global_timer_ns() - t0 < kWaitLimitNs) {
  }
}

inline bool ptr_aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// The caller's status words {code, detail}: the first error stays.
__device__ __forceinline__ void note_status(int32_t* status, int code, int detail) {
  if (status == nullptr) return;
  if (atomicCAS(status, PIQ_OK, code) == PIQ_OK) status[1] = detail;
}

// Whether [row0, row1) cannot be a sequence's rows in a tensor of `rows` rows.
__device__ __forceinline__ bool bad_rows(int64_t row0, int64_t row1, int64_t rows) {
  return row0 != row1 && (row0 < 0 || row1 < row0 || row1 > rows);
}

// Eight consecutive values of one row, as they lie in memory and in fp32.
template <typename T>
struct Eight {
  static constexpr int kVecs = sizeof(T) / 2;  // 16-byte vectors
  uint4 v[kVecs];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const;
};
template <>
__device__ __forceinline__ void Eight<float>::floats(float (&f)[8]) const {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(v[i].x);
    f[4 * i + 1] = __uint_as_float(v[i].y);
    f[4 * i + 2] = __uint_as_float(v[i].z);
    f[4 * i + 3] = __uint_as_float(v[i].w);
  }
}
template <>
__device__ __forceinline__ void Eight<__nv_bfloat16>::floats(float (&f)[8]) const {
  const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void Eight<__half>::floats(float (&f)[8]) const {
  const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

// Largest magnitude as a bit pattern: ordered like the values, and an infinity
// or NaN is larger than every finite one.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// scale = amax / 127 (0 below 2^-126, NaN for an infinity or NaN).
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  const float s = __fdiv_rn(__uint_as_float(amax_bits), 127.0f);
  return s < 1.17549435e-38f ? 0.0f : s;
}
// 0 for scales 0 and NaN, so that their codes are 0.
__device__ __forceinline__ float inverse_of(float scale) {
  return scale > 0.0f ? __frcp_rn(scale) : 0.0f;
}

// The largest magnitude of many runs of eight.  16-bit types are compared two at a
// time as integers.
template <typename T>
struct Largest {
  uint32_t v = 0;
  __device__ __forceinline__ void add(const Eight<T>& e) {
#pragma unroll
    for (int i = 0; i < Eight<T>::kVecs; ++i) {
      const uint32_t w[4] = {e.v[i].x, e.v[i].y, e.v[i].z, e.v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v = sizeof(T) == 2 ? __vmaxu2(v, w[j] & 0x7FFF7FFFu) : max(v, w[j] & 0x7FFFFFFFu);
    }
  }
  __device__ __forceinline__ uint32_t bits() const;  // of the fp32 value
};
template <>
__device__ __forceinline__ uint32_t Largest<float>::bits() const { return v; }
template <>
__device__ __forceinline__ uint32_t Largest<__nv_bfloat16>::bits() const {
  return max(v & 0xFFFFu, v >> 16) << 16;
}
template <>
__device__ __forceinline__ uint32_t Largest<__half>::bits() const {
  const uint32_t m = max(v & 0xFFFFu, v >> 16);
  return abs_bits(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
}

// rint(x * inverse) for |x| <= amax, in the low byte of each word: the product is
// at most 127 (1 + 2^-22), which needs no clipping, and adding 1.5 * 2^23 leaves the
// integer, rounded to nearest even, in the low bits of the sum (two's complement).
__device__ __forceinline__ uint32_t code_bits(float x, float inverse) {
  return __float_as_uint(__fadd_rn(__fmul_rn(x, inverse), 12582912.0f));
}
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// A non-finite x meets inverse 0 only, where every code is 0.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float inverse) {
  if (inverse == 0.0f) return make_uint2(0u, 0u);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = code_bits(f[i], inverse);
  return make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
}

// The sequence that ragged row `row` belongs to: the last b with cu[b] <= row,
// found by a whole warp, 32 starts a step; -1 when row < cu[0] or row >=
// cu[batch].  cu need not be valid: every index read lies in [0, batch].
__device__ __forceinline__ int find_sequence(const int32_t* cu, int batch, int64_t row, int lane) {
  int lo = 0, hi = batch + 1;  // answers lie in lo - 1 + (0 .. hi - lo)
  while (hi - lo > 0) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + step * lane + step - 1;  // the last of this lane's run
    const int probe = min(at, hi - 1);
    const bool le = __ldg(cu + probe) <= row;
    const unsigned votes = __ballot_sync(0xffffffffu, le);
    // runs are 0 .. 31; the first run whose last start is beyond `row` holds the border
    const int run = __ffs(~votes) - 1;
    if (run < 0) { lo = hi; break; }
    const int nlo = min(lo + step * run, hi);
    const int nhi = min(nlo + step - 1, hi);
    lo = nlo;
    hi = max(nhi, nlo);
    if (step == 1) { hi = lo; }
  }
  const int b = lo - 1;
  return (b < 0 || b >= batch) ? -1 : b;
}

}  // namespace piq
