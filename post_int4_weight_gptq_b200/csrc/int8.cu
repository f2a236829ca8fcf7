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
// TPR threads a row, each with up to four runs of eight values in registers:
// one pass over memory for rows of up to 32 TPR values, the rest of a longer
// row is read a second time.
constexpr int kRuns = 4;

template <typename T, int TPR>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
    quantize_rows_kernel(const T* __restrict__ X, int64_t rows, int64_t cols, int64_t ldx,
                         int8_t* __restrict__ codes, int64_t ldc, float* __restrict__ scales) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  constexpr int RPB = BLOCK / TPR;
  __shared__ uint32_t red[BLOCK / 32];
  pdl_wait();  // first: the product may then start on the weights once every CTA is here
  pdl_launch_dependents();
  const int tr = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / TPR;
  const bool live = row < rows;
  const T* x = X + (live ? row : 0) * ldx;
  const int64_t runs = live ? cols / 8 : 0;
  Eight<T> v[kRuns];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    const int64_t r = tr + static_cast<int64_t>(i) * TPR;
    if (r < runs)
      v[i].load(x + 8 * r);
    else
      v[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    float f[8];
    v[i].floats(f);
    m = amax_bits8(f, m);
  }
  for (int64_t r = tr + static_cast<int64_t>(kRuns) * TPR; r < runs; r += TPR) {
    Eight<T> e;
    float f[8];
    e.load(x + 8 * r);
    e.floats(f);
    m = amax_bits8(f, m);
  }
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
  if (cols <= 1024) {
    kern = quantize_rows_kernel<T, 32>;
    tpr = 32;
  } else if (cols <= 4096) {
    kern = quantize_rows_kernel<T, 128>;
    tpr = 128;
  } else if (cols <= 16384) {
    kern = quantize_rows_kernel<T, 512>;
    tpr = 512;
  } else {
    kern = quantize_rows_kernel<T, 1024>;
    tpr = 1024;
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

// Workspace: the codes of X (rows padded to 16 bytes) and its scales.
struct LinearWs {
  int64_t ldq;
  size_t scale_at, bytes;
};
LinearWs linear_ws(int64_t tokens, int64_t in) {
  LinearWs w;
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
      workspace == nullptr || !ptr_aligned(workspace, 256))
    return PIQ_ERR_INVALID_ARG;
  const LinearWs w = linear_ws(tokens, in);
  if (ws_bytes < w.bytes) return PIQ_ERR_WORKSPACE_TOO_SMALL;
  int rc = injected_fault();
  DeviceInfo info;
  if (rc == PIQ_OK) rc = device_info(&info);
  if (rc != PIQ_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int8_t* qx = static_cast<int8_t*>(workspace);
  float* sx = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.scale_at);
  rc = launch_quantize_rows(X, dtype, tokens, in, ldx, qx, w.ldq, sx, s);
  if (rc != PIQ_OK) return rc;
  return launch_int8_gemm(qx, w.ldq, sx, tokens, in, W, out, ldw, w_scale, bias, Y, dtype, ldy,
                          status, s);
}

}  // extern "C"
