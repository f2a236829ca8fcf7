// Linear layer on int8 codes: rows quantized to int8 with one scale each, and
// the matrix product of two such matrices.
//
//   Y[t, c] = (sum_k qx[t, k] qw[c, k]) sx[t] sw[c] + bias[c]
//
// Here the quantizer and the entry points; the product is int8_gemm.cu.
// The sum is exact in int32 (in <= 131064), so the result does not depend on
// the order or the split of the sum; the scales and the bias are applied in
// fp32 and the value is rounded once to Y's type.
#include <algorithm>

#include "serve.h"

namespace piq {

namespace {

// ------------------------------------------------------------ rows to int8
// TPR threads a row, each with up to eight runs of eight values in registers
// (four of fp32): one pass over memory for rows of up to 64 (32) TPR values, the
// rest of a longer row is read a second time.  Eight runs let two CTAs of 512
// threads share a multiprocessor on rows of 28672, one loading while the other
// reduces and stores; one CTA of 1024 took 1.5 times as long.
template <typename T>
constexpr int kRunsOf = sizeof(T) == 4 ? 4 : 8;

template <typename T, int TPR>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
    quantize_rows_kernel(const T* __restrict__ X, int64_t rows, int64_t cols, int64_t ldx,
                         int8_t* __restrict__ codes, int64_t ldc, float* __restrict__ scales) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  constexpr int RPB = BLOCK / TPR;
  constexpr int kRuns = kRunsOf<T>;
  __shared__ uint32_t red[BLOCK / 32];
  pdl_wait();  // first: the product may then start on the weights once every CTA is here
  pdl_launch_dependents();
  const int tr = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / TPR;
  const bool live = row < rows;
  const T* x = X + (live ? row : 0) * ldx;
  const int64_t runs = live ? cols / 8 : 0;
  Eight<T> v[kRuns];
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    const int64_t r = tr + static_cast<int64_t>(i) * TPR;
    if (r < runs)
      v[i].load(x + 8 * r);
    else
      v[i].zero();
  }
  Largest<T> top;
#pragma unroll
  for (int i = 0; i < kRuns; ++i) top.add(v[i]);
  for (int64_t r = tr + static_cast<int64_t>(kRuns) * TPR; r < runs; r += TPR) {
    Eight<T> e;
    e.load(x + 8 * r);
    top.add(e);
  }
  uint32_t m = top.bits();
  m = __reduce_max_sync(0xffffffffu, m);
  if (TPR > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    const int w0 = (threadIdx.x / TPR) * (TPR / 32);
    m = red[w0 + (threadIdx.x & 31) % (TPR / 32)];
    m = __reduce_max_sync(0xffffffffu, m);
  }
  const float scale = scale_of(m);
  const float inv = inverse_of(scale);
  if (live && tr == 0) scales[row] = scale;
  int8_t* c = codes + (live ? row : 0) * ldc;
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    const int64_t r = tr + static_cast<int64_t>(i) * TPR;
    if (r < runs) {
      float f[8];
      v[i].floats(f);
      *reinterpret_cast<uint2*>(c + 8 * r) = codes8(f, inv);
    }
  }
  for (int64_t r = tr + static_cast<int64_t>(kRuns) * TPR; r < runs; r += TPR) {
    Eight<T> e;
    float f[8];
    e.load(x + 8 * r);
    e.floats(f);
    *reinterpret_cast<uint2*>(c + 8 * r) = codes8(f, inv);
  }
}

template <typename T>
int launch_quantize_rows_t(const T* X, int64_t rows, int64_t cols, int64_t ldx, int8_t* codes,
                           int64_t ldc, float* scales, cudaStream_t stream) {
  void (*kern)(const T*, int64_t, int64_t, int64_t, int8_t*, int64_t, float*) = nullptr;
  int tpr = 0;
  const int64_t per_thread = 8 * kRunsOf<T>;
  if (cols <= 32 * per_thread) {
    kern = quantize_rows_kernel<T, 32>;
    tpr = 32;
  } else if (cols <= 128 * per_thread) {
    kern = quantize_rows_kernel<T, 128>;
    tpr = 128;
  } else if (cols <= 256 * per_thread) {
    kern = quantize_rows_kernel<T, 256>;
    tpr = 256;
  } else {
    kern = quantize_rows_kernel<T, 512>;
    tpr = 512;
  }
  const int block = std::max(tpr, 256);
  const int64_t grid = ceil_div(rows, block / tpr);
  note_launch();
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(block), 0, stream, X, rows, cols,
                    ldx, codes, ldc, scales) == cudaSuccess
             ? PIQ_OK
             : PIQ_ERR_CUDA;
}

int launch_quantize_rows(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                         int8_t* codes, int64_t ldc, float* scales, cudaStream_t stream) {
  switch (dtype) {
    case PIQ_BF16:
      return launch_quantize_rows_t(static_cast<const __nv_bfloat16*>(X), rows, cols, ldx, codes,
                                    ldc, scales, stream);
    case PIQ_FP16:
      return launch_quantize_rows_t(static_cast<const __half*>(X), rows, cols, ldx, codes, ldc,
                                    scales, stream);
    default:
      return launch_quantize_rows_t(static_cast<const float*>(X), rows, cols, ldx, codes, ldc,
                                    scales, stream);
  }
}

// ------------------------------------------------------- a few tokens, one kernel
// A warp takes one output channel: its weights stream through registers in 16-byte
// pieces (4 KB a warp under way), asked for before anything else, so that the wait
// for them covers the quantization of the tokens, which every CTA does for itself
// into shared memory (a token is 2 in bytes from L2).  One launch, no workspace.
// Bound by the weights' bytes where they are many, by the launch and one trip to
// memory where they are few: one token, 4096 -> 4096, took 7.3 us as two kernels.
constexpr int kFewWarps = 8;
constexpr int kPieces = 8;  // 16-byte weight pieces a lane has under way

template <typename T, int TOK>
__global__ void __launch_bounds__(32 * kFewWarps)
    int8_few_kernel(const T* __restrict__ X, int tokens, int in, int64_t ldx,
                    const int8_t* __restrict__ W, int64_t out, int64_t ldw,
                    const float* __restrict__ sw, const float* __restrict__ bias,
                    T* __restrict__ Y, int64_t ldy) {
  extern __shared__ __align__(16) int8_t codes[];  // [TOK][row], zeros behind `in`
  __shared__ uint32_t red[TOK][kFewWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = (in + 15) & ~15;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kFewWarps + warp;
  pdl_launch_dependents();
  pdl_wait();
  const int8_t* w = W + (c < out ? c : 0) * ldw;
  auto load = [&](int k) {
    if (k + 16 <= in) return __ldg(reinterpret_cast<const uint4*>(w + k));
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (k < in) {  // in is a multiple of 8
      const uint2 h = __ldg(reinterpret_cast<const uint2*>(w + k));
      v.x = h.x;
      v.y = h.y;
    }
    return v;
  };
  uint4 a[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) a[i] = load(16 * lane + 512 * i);
  const float sc = c < out ? __ldg(sw + c) : 0.0f;
  const float bc = bias != nullptr && c < out ? __ldg(bias + c) : 0.0f;

  Largest<T> top[TOK];
  for (int k = 8 * threadIdx.x; k < in; k += 8 * 32 * kFewWarps)
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
      Eight<T> e;
      e.load(X + min(t, tokens - 1) * ldx + k);
      top[t].add(e);
    }
#pragma unroll
  for (int t = 0; t < TOK; ++t) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, top[t].bits());
    if (lane == 0) red[t][warp] = m;
  }
  __syncthreads();
  float scale[TOK], inv[TOK];
#pragma unroll
  for (int t = 0; t < TOK; ++t) {
    scale[t] = scale_of(__reduce_max_sync(0xffffffffu, red[t][lane % kFewWarps]));
    inv[t] = inverse_of(scale[t]);
  }
  for (int k = 8 * threadIdx.x; k < row; k += 8 * 32 * kFewWarps)
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
      uint2 q = make_uint2(0u, 0u);
      if (k < in) {
        Eight<T> e;
        float f[8];
        e.load(X + min(t, tokens - 1) * ldx + k);
        e.floats(f);
        q = codes8(f, inv[t]);
      }
      *reinterpret_cast<uint2*>(codes + t * row + k) = q;
    }
  __syncthreads();

  int acc[TOK] = {};
  for (int k0 = 0; k0 < in; k0 += 512 * kPieces) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int k = k0 + 16 * lane + 512 * i;
      if (k >= in) break;
#pragma unroll
      for (int t = 0; t < TOK; ++t) {
        const uint4 b = *reinterpret_cast<const uint4*>(codes + t * row + k);
        acc[t] = __dp4a(static_cast<int>(a[i].x), static_cast<int>(b.x), acc[t]);
        acc[t] = __dp4a(static_cast<int>(a[i].y), static_cast<int>(b.y), acc[t]);
        acc[t] = __dp4a(static_cast<int>(a[i].z), static_cast<int>(b.z), acc[t]);
        acc[t] = __dp4a(static_cast<int>(a[i].w), static_cast<int>(b.w), acc[t]);
      }
      a[i] = load(k + 512 * kPieces);
    }
  }
#pragma unroll
  for (int t = 0; t < TOK; ++t) {
    acc[t] = __reduce_add_sync(0xffffffffu, acc[t]);
    if (lane == t && t < tokens && c < out)
      Y[t * ldy + c] = from_float<T>(fmaf(static_cast<float>(acc[t]) * scale[t], sc, bc));
  }
}

// Tokens that the kernel above takes: its CTAs all quantize them, which stops
// paying when that reads as much as a CTA's weights.
constexpr int64_t kFewTokens = 1, kFewValues = 16384;
bool few_tokens(int64_t tokens, int64_t in) {
  return tokens <= kFewTokens && tokens * in <= kFewValues;
}

template <typename T>
int launch_few_t(const T* X, int64_t tokens, int64_t in, int64_t ldx, const int8_t* W, int64_t out,
                 int64_t ldw, const float* sw, const float* bias, T* Y, int64_t ldy,
                 cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(ceil_div(out, kFewWarps));
  const int tok = tokens == 1 ? 1 : tokens == 2 ? 2 : 4;
  const size_t smem = static_cast<size_t>(tok) * ((in + 15) / 16 * 16);  // at most 32 KB
  auto kern = tok == 1 ? int8_few_kernel<T, 1> : tok == 2 ? int8_few_kernel<T, 2>
                                                          : int8_few_kernel<T, 4>;
  note_launch();
  return launch_pdl(kern, dim3(grid), dim3(32 * kFewWarps), smem, stream, X,
                    static_cast<int>(tokens), static_cast<int>(in), ldx, W, out, ldw, sw, bias, Y,
                    ldy) == cudaSuccess
             ? PIQ_OK
             : PIQ_ERR_CUDA;
}

// Workspace: the codes of X (rows padded to 16 bytes) and its scales.
struct LinearWs {
  int64_t ldq;
  size_t scale_at, bytes;
};
LinearWs linear_ws(int64_t tokens, int64_t in) {
  LinearWs w;
  if (few_tokens(tokens, in)) return LinearWs{0, 0, 0};
  w.ldq = (in + 15) / 16 * 16;
  w.scale_at = (static_cast<size_t>(std::max<int64_t>(tokens, 1)) * w.ldq + 255) / 256 * 256;
  w.bytes = w.scale_at + (static_cast<size_t>(std::max<int64_t>(tokens, 1)) * 4 + 255) / 256 * 256;
  return w;
}

bool linear_sizes_ok(int64_t tokens, int64_t out, int64_t in) {
  return tokens >= 0 && tokens <= (int64_t)1 << 30 && out >= 1 && out <= (int64_t)1 << 24 &&
         in >= 8 && in % 8 == 0 && in <= kInt8MaxIn;
}

}  // namespace
}  // namespace piq

extern "C" {
using namespace piq;

int piq_int8_quantize_rows(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                           int8_t* codes, int64_t ldc, float* scales, void* stream) {
  if (dtype < PIQ_BF16 || dtype > PIQ_FP32 || rows < 0 || rows > (int64_t)1 << 30 || cols < 8 ||
      cols % 8 != 0 || cols > (int64_t)1 << 20 || ldx < cols || ldx % 8 != 0 || ldc < cols ||
      ldc % 8 != 0)
    return PIQ_ERR_INVALID_ARG;
  if (rows == 0) return PIQ_OK;
  if (X == nullptr || codes == nullptr || scales == nullptr || !ptr_aligned(X, 16) ||
      !ptr_aligned(codes, 8) || !ptr_aligned(scales, 4))
    return PIQ_ERR_INVALID_ARG;
  int rc = injected_fault();
  DeviceInfo info;
  if (rc == PIQ_OK) rc = device_info(&info);
  if (rc != PIQ_OK) return rc;
  return launch_quantize_rows(X, dtype, rows, cols, ldx, codes, ldc, scales,
                              static_cast<cudaStream_t>(stream));
}

int piq_int8_linear_workspace_bytes(int64_t tokens, int64_t out, int64_t in, size_t* bytes) {
  if (bytes == nullptr || !linear_sizes_ok(tokens, out, in)) return PIQ_ERR_INVALID_ARG;
  *bytes = linear_ws(tokens, in).bytes;
  return PIQ_OK;
}

int piq_int8_linear(const void* X, int dtype, int64_t tokens, int64_t in, int64_t ldx,
                    const int8_t* W, int64_t out, int64_t ldw, const float* w_scale,
                    const float* bias, void* Y, int64_t ldy, int32_t* status, void* workspace,
                    size_t ws_bytes, void* stream) {
  if (dtype < PIQ_BF16 || dtype > PIQ_FP32 || !linear_sizes_ok(tokens, out, in) || ldx < in ||
      ldx % 8 != 0 || ldw < in || ldw % 16 != 0 || ldy < out)
    return PIQ_ERR_INVALID_ARG;
  if (tokens == 0) return PIQ_OK;
  if (X == nullptr || W == nullptr || w_scale == nullptr || Y == nullptr || !ptr_aligned(X, 16) ||
      !ptr_aligned(W, 16) || !ptr_aligned(w_scale, 4) || !ptr_aligned(bias, 4) ||
      !ptr_aligned(Y, dtype == PIQ_FP32 ? 4 : 2) || !ptr_aligned(status, 4) ||
      (workspace == nullptr && !few_tokens(tokens, in)) || !ptr_aligned(workspace, 256))
    return PIQ_ERR_INVALID_ARG;
  const LinearWs w = linear_ws(tokens, in);
  if (ws_bytes < w.bytes) return PIQ_ERR_WORKSPACE_TOO_SMALL;
  int rc = injected_fault();
  DeviceInfo info;
  if (rc == PIQ_OK) rc = device_info(&info);
  if (rc != PIQ_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (few_tokens(tokens, in)) {
    switch (dtype) {
      case PIQ_BF16:
        return launch_few_t(static_cast<const __nv_bfloat16*>(X), tokens, in, ldx, W, out, ldw,
                            w_scale, bias, static_cast<__nv_bfloat16*>(Y), ldy, s);
      case PIQ_FP16:
        return launch_few_t(static_cast<const __half*>(X), tokens, in, ldx, W, out, ldw, w_scale,
                            bias, static_cast<__half*>(Y), ldy, s);
      default:
        return launch_few_t(static_cast<const float*>(X), tokens, in, ldx, W, out, ldw, w_scale,
                            bias, static_cast<float*>(Y), ldy, s);
    }
  }
  int8_t* qx = static_cast<int8_t*>(workspace);
  float* sx = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.scale_at);
  rc = launch_quantize_rows(X, dtype, tokens, in, ldx, qx, w.ldq, sx, s);
  if (rc != PIQ_OK) return rc;
  return launch_int8_gemm(qx, w.ldq, sx, tokens, in, W, out, ldw, w_scale, bias, Y, dtype, ldy,
                          status, s);
}

}  // extern "C"
