// Shared by the two attention kernels over the 8-bit cache (kv8_attn.cu: few
// rows, kv8_prompt.cu: many).
#pragma once

#include "serve.h"

namespace piq {

struct Kv8Attn {
  const void* q;
  int64_t tokens, ldq;
  const int32_t *cu, *lens;
  const int32_t* table;
  int64_t width, ldt;
  const int8_t *kc, *vc;
  const float *ks, *vs;
  int64_t pages;
  int batch, heads, kv_heads, block, group;  // group = heads / kv_heads
  float scale2;                              // scale * log2(e)
  int window;                                // 0: none
  int64_t max_new, max_len;
  int chunk;                                 // keys a CTA, a multiple of 128
  int chunks;                                // most chunks of a sequence
  void* out;
  int64_t ldo;
  float* lse;
  float* part_o;   // [chunks][tokens][heads][D] when chunks > 1: each chunk's own average
  float2* part_ml; // [chunks][tokens][heads]: running maximum (log2), sum
  int32_t* status;
  uint64_t wait_ns;  // limit of a wait
  uint32_t low_bytes = 0x00FF00FFu;  // a parameter, so that (w & mask) ^ constant is one
                                     // instruction: with two literals it became two
};

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLow = -3.0e38f;      // below every score: "no key yet"
constexpr float kSlack = 7.0f;        // log2 by which a score may pass the maximum

// The weights of the values enter the second product in fp16 as 2^(x - m) v_scale c.
// c = 2^(7 - d) is a row's own: 2^d is the power of two at or below the largest v_scale
// of the blocks that the row has seen keys of, so that what a row does not see takes no
// bits from it.  d is at least -119 and c a normal number; with scores up to kSlack above
// the maximum a weight stays below 2^15.
constexpr float kFirstFactor = 0x1p126f;
constexpr float kWide = 256.0f;  // v_scale c from which c has to move

// The factor of a row that had c and sees a block of scale vs >= 0.
__device__ __forceinline__ float factor_for(float c, float vs) {
  const int d = max(static_cast<int>(__float_as_uint(vs) >> 23) - 127, -119);
  return fminf(c, __uint_as_float(static_cast<uint32_t>(134 - d) << 23));
}
__device__ __forceinline__ int shift_of(float c) {  // d
  return 134 - static_cast<int>(__float_as_uint(c) >> 23);
}
__device__ __forceinline__ float undo_factor(int d) {  // 1 / c = 2^(d - 7)
  return __uint_as_float(static_cast<uint32_t>(120 + d) << 23);
}

// The block in which the first key that some query sees lies: chunks are counted
// from its start.  (Lengths are at most 2^26 and rows below 2^31, so positions are
// 32-bit numbers; 64-bit divisions cost these kernels thousands of cycles.)
__device__ __forceinline__ int first_block_key(int len, int n, int window, int block) {
  return window > 0 ? max(0, len - n + 1 - window) & -block : 0;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}

// A row of q in fp16 and the factor that undoes its scaling.  bf16 rows are
// scaled by the power of two that brings their largest magnitude into [1, 2).
template <typename T>
__device__ __forceinline__ float row_exponent(float amax, float& mul);
template <>
__device__ __forceinline__ float row_exponent<__half>(float amax, float& mul) {
  mul = 1.0f;
  return amax < __uint_as_float(0x7F800000u) ? 1.0f : __uint_as_float(0x7FC00000u);
}
template <>
__device__ __forceinline__ float row_exponent<__nv_bfloat16>(float amax, float& mul) {
  const uint32_t e = __float_as_uint(amax) >> 23;  // biased exponent
  if (e == 255u || !(amax == amax)) {
    mul = 0.0f;
    return __uint_as_float(0x7FC00000u);
  }
  if (e < 2u || e > 252u) {  // mul and its inverse stay normal numbers
    const bool big = e > 252u;
    mul = big ? 0x1p-126f : 0x1p126f;
    return big ? 0x1p126f : 0x1p-126f;
  }
  mul = __uint_as_float((254u - e) << 23);
  return __uint_as_float(e << 23);
}

// Whether the lengths of a sequence (of any rows) cannot be.
__device__ __forceinline__ bool bad_lengths(const Kv8Attn& p, int64_t q0, int64_t q1,
                                            int64_t len) {
  const int64_t n = q1 - q0;
  return bad_rows(q0, q1, p.tokens) ||
         (n != 0 && (n > p.max_new || len < n || len > p.max_len || len > p.width * p.block));
}
// Then one CTA, all of it, sets the status and the rows, as far as they exist, to NaN.
template <typename T, int D>
__device__ __forceinline__ void report_lengths(const Kv8Attn& p, int b, int64_t q0, int64_t q1) {
  if (threadIdx.x == 0) note_status(p.status, PIQ_ERR_INVALID_ARG, b);
  const int64_t t0 = max(q0, static_cast<int64_t>(0)), t1 = min(q1, p.tokens);
  const float nan = __uint_as_float(0x7FC00000u);
  for (int64_t t = t0; t < t1; ++t) {
    for (int i = threadIdx.x; i < p.heads * D; i += blockDim.x)
      static_cast<T*>(p.out)[t * p.ldo + i] = from_float<T>(nan);
    if (p.lse != nullptr)
      for (int i = threadIdx.x; i < p.heads; i += blockDim.x) p.lse[t * p.heads + i] = nan;
  }
}

// kv8_prompt.cu: the chunk kernel for many rows a kv head.
constexpr int kPromptRows = 256;  // query rows a CTA
template <typename T, int D>
int launch_prompt(const Kv8Attn& p, cudaStream_t stream);

}  // namespace piq
