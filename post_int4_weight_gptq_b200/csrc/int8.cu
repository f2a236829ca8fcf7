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
#include <atomic>

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

// ----------------------------------------------------------- one token, one kernel
// A warp takes one output channel: its weights stream through registers in 16-byte
// pieces (4 KB a warp under way), asked for before anything else, so that the wait
// for them covers the quantization of the token, which every CTA does for itself into
// shared memory (2 in bytes from L2).  One launch, no workspace.  Bound by the launch
// and one trip to memory: 4.5 us for 4096 -> 4096 (3.7 TB/s), 7.0 us as two kernels.
// More tokens gain nothing by it (two kernels second, in us): 2 tokens 7.3 and 6.8-7.0,
// 4 tokens 10.5 and 7.0, 4 from 4096 to 11008 23.0 and 13.3: all CTAs quantize all
// tokens, and a weight piece meets as many pieces of codes in shared memory.
constexpr int kOneWarps = 8;
constexpr int kPieces = 8;  // 16-byte weight pieces a lane has under way

template <typename T>
__global__ void __launch_bounds__(32 * kOneWarps)
    int8_one_kernel(const T* __restrict__ X, int in, const int8_t* __restrict__ W, int64_t out,
                    int64_t ldw, const float* __restrict__ sw, const float* __restrict__ bias,
                    T* __restrict__ Y) {
  extern __shared__ __align__(16) int8_t codes[];  // `in` padded to 16 with zeros
  __shared__ uint32_t red[kOneWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = (in + 15) & ~15;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kOneWarps + warp;
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

  Largest<T> top;
  for (int k = 8 * threadIdx.x; k < in; k += 8 * 32 * kOneWarps) {
    Eight<T> e;
    e.load(X + k);
    top.add(e);
  }
  const uint32_t m = __reduce_max_sync(0xffffffffu, top.bits());
  if (lane == 0) red[warp] = m;
  __syncthreads();
  const float scale = scale_of(__reduce_max_sync(0xffffffffu, red[lane % kOneWarps]));
  const float inv = inverse_of(scale);
  for (int k = 8 * threadIdx.x; k < row; k += 8 * 32 * kOneWarps) {
    uint2 q = make_uint2(0u, 0u);
    if (k < in) {
      Eight<T> e;
      float f[8];
      e.load(X + k);
      e.floats(f);
      q = codes8(f, inv);
    }
    *reinterpret_cast<uint2*>(codes + k) = q;
  }
  __syncthreads();

  int acc = 0;
  for (int k0 = 0; k0 < in; k0 += 512 * kPieces) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int k = k0 + 16 * lane + 512 * i;
      if (k >= in) break;
      const uint4 b = *reinterpret_cast<const uint4*>(codes + k);
      acc = __dp4a(static_cast<int>(a[i].x), static_cast<int>(b.x), acc);
      acc = __dp4a(static_cast<int>(a[i].y), static_cast<int>(b.y), acc);
      acc = __dp4a(static_cast<int>(a[i].z), static_cast<int>(b.z), acc);
      acc = __dp4a(static_cast<int>(a[i].w), static_cast<int>(b.w), acc);
      a[i] = load(k + 512 * kPieces);
    }
  }
  acc = __reduce_add_sync(0xffffffffu, acc);
  if (lane == 0 && c < out) Y[c] = from_float<T>(fmaf(static_cast<float>(acc) * scale, sc, bc));
}

// What the kernel above takes: at 16384 -> 4096 the two ways meet (15.5 and 15.7 us).
constexpr int64_t kOneValues = 16384;
bool one_kernel(int64_t tokens, int64_t in) { return tokens == 1 && in <= kOneValues; }

template <typename T>
int launch_one_t(const T* X, int64_t in, const int8_t* W, int64_t out, int64_t ldw,
                 const float* sw, const float* bias, T* Y, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(ceil_div(out, kOneWarps));
  const size_t smem = static_cast<size_t>((in + 15) / 16 * 16);
  note_launch();
  return launch_pdl(int8_one_kernel<T>, dim3(grid), dim3(32 * kOneWarps), smem, stream, X,
                    static_cast<int>(in), W, out, ldw, sw, bias, Y) == cudaSuccess
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
  if (one_kernel(tokens, in)) return LinearWs{0, 0, 0};
  w.ldq = (in + 15) / 16 * 16;
  w.scale_at = (static_cast<size_t>(std::max<int64_t>(tokens, 1)) * w.ldq + 255) / 256 * 256;
  w.bytes = w.scale_at + (static_cast<size_t>(std::max<int64_t>(tokens, 1)) * 4 + 255) / 256 * 256;
  return w;
}

std::atomic<uint64_t> g_wait_ns{kWaitLimitNs};

bool linear_sizes_ok(int64_t tokens, int64_t out, int64_t in) {
  return tokens >= 0 && tokens <= (int64_t)1 << 30 && out >= 1 && out <= (int64_t)1 << 24 &&
         in >= 8 && in % 8 == 0 && in <= kInt8MaxIn;
}

}  // namespace

uint64_t serving_wait_ns() { return g_wait_ns.load(std::memory_order_relaxed); }

}  // namespace piq

extern "C" {
using namespace piq;

int piq_serving_wait_limit(uint64_t wait_ns) {
  if (wait_ns > 10000000000ull) return PIQ_ERR_INVALID_ARG;
  g_wait_ns.store(wait_ns == 0 ? kWaitLimitNs : wait_ns, std::memory_order_relaxed);
  return PIQ_OK;
}

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
      (workspace == nullptr && !one_kernel(tokens, in)) || !ptr_aligned(workspace, 256))
    return PIQ_ERR_INVALID_ARG;
  const LinearWs w = linear_ws(tokens, in);
  if (ws_bytes < w.bytes) return PIQ_ERR_WORKSPACE_TOO_SMALL;
  int rc = injected_fault();
  DeviceInfo info;
  if (rc == PIQ_OK) rc = device_info(&info);
  if (rc != PIQ_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (one_kernel(tokens, in)) {
    switch (dtype) {
      case PIQ_BF16:
        return launch_one_t(static_cast<const __nv_bfloat16*>(X), in, W, out, ldw, w_scale, bias,
                            static_cast<__nv_bfloat16*>(Y), s);
      case PIQ_FP16:
        return launch_one_t(static_cast<const __half*>(X), in, W, out, ldw, w_scale, bias,
                            static_cast<__half*>(Y), s);
      default:
        return launch_one_t(static_cast<const float*>(X), in, W, out, ldw, w_scale, bias,
                            static_cast<float*>(Y), s);
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
