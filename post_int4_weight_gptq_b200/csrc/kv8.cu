// The 8-bit paged key/value cache: quantization of keys and values as they are
// written, and reading them back.  One scale for each block of tokens and head:
//
//   scale = max(scale so far, amax(new values of the block) / 127)
//   code  = rint(x / scale), codes already there: rint(c * old / new)
//
// Both are bound by memory: a byte out for every value in, or the reverse.
#include <algorithm>

#include "serve.h"

namespace piq {
namespace {

struct Kv8Write {
  const void *k, *v;
  int64_t tokens, ldk, ldv;
  const int32_t *cu, *lens;
  const int32_t* table;
  int64_t width, ldt;
  int8_t *kc, *vc;
  float *ks, *vs;
  int64_t pages;
  int batch, heads, block;
  int32_t* status;
};

// Work items are (sequence, block) pairs numbered without knowing the lengths on
// the host: a run of n tokens spans at most floor(n / block) + 2 blocks, so
// sequence b's items start at floor(cu[b] / block) + 2 b and the last item is
// below floor(tokens / block) + 2 batch.  floor_start is what is searched.
__device__ __forceinline__ int64_t item_start(const int32_t* cu, int b, int block) {
  return __ldg(cu + b) / block + 2 * static_cast<int64_t>(b);
}

// The last sequence whose items start at or before `item`, by a whole warp.
__device__ __forceinline__ int find_item(const int32_t* cu, int batch, int block, int64_t item,
                                         int lane) {
  int lo = 0, hi = batch;
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int probe = min(lo + step * lane + step - 1, hi - 1);
    const unsigned votes =
        __ballot_sync(0xffffffffu, item_start(cu, probe, block) <= item);
    const int run = __ffs(~votes) - 1;
    if (run < 0) {
      lo = hi;
      break;
    }
    const int nlo = min(lo + step * run, hi);
    hi = min(nlo + step - 1, hi);
    lo = nlo;
  }
  return lo - 1;
}

// One block of tokens of one head, keys (blockIdx.z == 0) or values (1).
// NR > 0: NR runs of eight values a thread, the whole block read once, its scale
// found by a reduction over the CTA, codes written from the registers.
// NR == 0, for calls of a few tokens a sequence: only the new tokens' runs are
// visited, twice (the second time from the cache), in few registers, so that the
// CTAs of a decoding step fit the machine at once.
// The tokens are asked for before the page they go to is looked up.
template <typename T, int D, int NR>
__global__ void __launch_bounds__(256) kv8_append_kernel(Kv8Write p) {
  constexpr int RPT = D / 8;  // runs a token
  __shared__ uint32_t red[8];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int head = blockIdx.y;
  auto bad = [&](int64_t row0, int64_t row1, int64_t before) {
    return bad_rows(row0, row1, p.tokens) ||
           (row0 != row1 && (before < 0 || before + (row1 - row0) > p.width * p.block));
  };
  // Bad lengths are reported by a CTA of its own (one item more than there can be), for the
  // whole batch: with starts that cannot be, the search may pass a sequence by.
  if (blockIdx.x == gridDim.x - 1) {
    if (head == 0 && blockIdx.z == 0)
      for (int i = threadIdx.x; i < p.batch; i += blockDim.x)
        if (bad(__ldg(p.cu + i), __ldg(p.cu + i + 1), __ldg(p.lens + i)))
          note_status(p.status, PIQ_ERR_INVALID_ARG, i);
    return;
  }
  const int b = find_item(p.cu, p.batch, p.block, blockIdx.x, lane);
  if (b < 0) return;
  const int64_t row0 = __ldg(p.cu + b), row1 = __ldg(p.cu + b + 1);
  const int64_t before = __ldg(p.lens + b);
  if (row0 == row1 || bad(row0, row1, before)) return;
  const int shift = __ffs(p.block) - 1;
  const int64_t blk = (before >> shift) + (blockIdx.x - item_start(p.cu, b, p.block));
  const int64_t base = blk << shift;               // position of the block's first token
  const int64_t end = before + (row1 - row0);      // the sequence's tokens after this call
  if (base >= end) return;
  const int o0 = static_cast<int>(max(before, base) - base);         // first new token
  const int o1 = static_cast<int>(min(end, base + p.block) - base);  // behind the last one
  const bool vals = blockIdx.z != 0;
  const int64_t ld = vals ? p.ldv : p.ldk;
  const T* src = static_cast<const T*>(vals ? p.v : p.k) +
                 (row0 + (base - before)) * ld + head * D;  // the block's token 0, if it is new

  Eight<T> v[NR > 0 ? NR : 1];
  Largest<T> top;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int run = threadIdx.x + i * blockDim.x;
    const int o = run / RPT;
    if (o >= o0 && o < o1)
      v[i].load(src + o * ld + (run % RPT) * 8);
    else
      v[i].zero();
  }
  const int64_t page = __ldg(p.table + b * p.ldt + blk);
  if (page < 0 || page >= p.pages) {
    if (threadIdx.x == 0) note_status(p.status, PIQ_ERR_INVALID_ARG, b);
    return;
  }
  int8_t* dst = (vals ? p.vc : p.kc) + (page * p.heads + head) * p.block * static_cast<int64_t>(D);
  float* sp = (vals ? p.vs : p.ks) + page * p.heads + head;
  const float old = o0 > 0 ? *sp : 0.0f;  // read before thread 0 writes it, below the barrier
  if (NR > 0) {
#pragma unroll
    for (int i = 0; i < NR; ++i) top.add(v[i]);
  } else {
    for (int run = o0 * RPT + threadIdx.x; run < o1 * RPT; run += blockDim.x) {
      v[0].load(src + (run / RPT) * ld + (run % RPT) * 8);
      top.add(v[0]);
    }
  }
  uint32_t m = __reduce_max_sync(0xffffffffu, top.bits());
  if (lane == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = red[lane % (blockDim.x / 32)];
  m = __reduce_max_sync(0xffffffffu, m);
  float scale = scale_of(m);
  if (!(scale >= old) && scale == scale) scale = old;  // the larger one; NaN of either stays
  const float inv = inverse_of(scale);
  if (threadIdx.x == 0) *sp = scale;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int run = threadIdx.x + i * blockDim.x;
    const int o = run / RPT;
    if (o >= o0 && o < o1) {
      float f[8];
      v[i].floats(f);
      *reinterpret_cast<uint2*>(dst + run * 8) = codes8(f, inv);
    }
  }
  if (NR == 0)
    for (int run = o0 * RPT + threadIdx.x; run < o1 * RPT; run += blockDim.x) {
      float f[8];
      v[0].load(src + (run / RPT) * ld + (run % RPT) * 8);
      v[0].floats(f);
      *reinterpret_cast<uint2*>(dst + run * 8) = codes8(f, inv);
    }
  // codes already there: unchanged while the scale is
  if (o0 > 0 && !(scale == old)) {
    const float ratio = scale > 0.0f ? __fdiv_rn(old, scale) : 0.0f;
    for (int run = threadIdx.x; run < o0 * RPT; run += blockDim.x) {
      const uint2 c = *reinterpret_cast<const uint2*>(dst + run * 8);
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[j] = static_cast<float>(static_cast<int8_t>(c.x >> (8 * j)));
        f[4 + j] = static_cast<float>(static_cast<int8_t>(c.y >> (8 * j)));
      }
      *reinterpret_cast<uint2*>(dst + run * 8) = codes8(f, ratio);
    }
  }
}

struct Kv8Read {
  const int8_t *kc, *vc;
  const float *ks, *vs;
  int64_t pages;
  int heads, block;
  const int32_t *cu, *start;
  int batch;
  const int32_t* table;
  int64_t width, ldt, rows;
  void *k, *v;
  int64_t ldk, ldv;
  int32_t* status;
};

// One warp a row of the output: all heads of one token, keys or values.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv8_read_kernel(Kv8Read p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  // starts that no row may lead to: a CTA behind those with rows looks at the whole batch
  if (blockIdx.x == gridDim.x - 1 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < p.batch; i += blockDim.x)
      if (bad_rows(__ldg(p.cu + i), __ldg(p.cu + i + 1), p.rows))
        note_status(p.status, PIQ_ERR_INVALID_ARG, i);
  if (row >= p.rows) return;
  const int b = find_sequence(p.cu, p.batch, row, lane);
  if (b < 0) return;
  const int64_t row0 = __ldg(p.cu + b), row1 = __ldg(p.cu + b + 1);
  const int64_t pos = __ldg(p.start + b) + (row - row0);
  int64_t page = -1;
  const int shift = __ffs(p.block) - 1;
  if (pos >= 0 && pos < p.width * p.block && !bad_rows(row0, row1, p.rows))
    page = __ldg(p.table + b * p.ldt + (pos >> shift));
  const bool bad = page < 0 || page >= p.pages;
  if (bad && lane == 0) note_status(p.status, PIQ_ERR_INVALID_ARG, b);
  const bool vals = blockIdx.y != 0;
  const int8_t* codes = vals ? p.vc : p.kc;
  const float* scales = vals ? p.vs : p.ks;
  T* out = static_cast<T*>(vals ? p.v : p.k) + row * (vals ? p.ldv : p.ldk);
  const int off = static_cast<int>(pos) & (p.block - 1);
  for (int run = lane; run < p.heads * (D / 8); run += 32) {
    const int head = run / (D / 8), d = (run % (D / 8)) * 8;
    uint2 c = make_uint2(0u, 0u);
    float s = __uint_as_float(0x7FC00000u);
    if (!bad) {
      c = __ldg(reinterpret_cast<const uint2*>(
          codes + ((page * p.heads + head) * p.block + off) * static_cast<int64_t>(D) + d));
      s = __ldg(scales + page * p.heads + head);
    }
    Eight<T> e;
    T* w = reinterpret_cast<T*>(e.v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = from_float<T>(static_cast<float>(static_cast<int8_t>(c.x >> (8 * j))) * s);
      w[4 + j] = from_float<T>(static_cast<float>(static_cast<int8_t>(c.y >> (8 * j))) * s);
    }
#pragma unroll
    for (int i = 0; i < Eight<T>::kVecs; ++i)
      reinterpret_cast<uint4*>(out + run * 8)[i] = e.v[i];
  }
}

// New tokens a sequence, on average, up to which most of a block is not new.
constexpr int64_t kFewNew = 4;

template <typename T, int D>
int launch_append(const Kv8Write& p, cudaStream_t stream) {
  const int runs = p.block * (D / 8);  // 128 .. 2048
  const bool few = p.tokens <= kFewNew * p.batch;
  const int threads = !few && runs > 1024 ? 256 : 128;
  void (*kern)(Kv8Write) = nullptr;
  switch (few ? 0 : runs / threads) {
    case 0: kern = kv8_append_kernel<T, D, 0>; break;
    case 1: kern = kv8_append_kernel<T, D, 1>; break;
    case 2: kern = kv8_append_kernel<T, D, 2>; break;
    case 4: kern = kv8_append_kernel<T, D, 4>; break;
    default: kern = kv8_append_kernel<T, D, 8>; break;
  }
  const int64_t items = p.tokens / p.block + 2 * static_cast<int64_t>(p.batch);
  note_launch();
  return launch_pdl(kern, dim3(static_cast<unsigned>(items + 1), p.heads, 2), dim3(threads), 0,
                    stream, p) == cudaSuccess
             ? PIQ_OK
             : PIQ_ERR_CUDA;
}

template <typename T, int D>
int launch_read(const Kv8Read& p, cudaStream_t stream) {
  note_launch();
  return launch_pdl(kv8_read_kernel<T, D>, dim3(static_cast<unsigned>(ceil_div(p.rows, 8) + 1), 2),
                    dim3(256), 0, stream, p) == cudaSuccess
             ? PIQ_OK
             : PIQ_ERR_CUDA;
}

}  // namespace

bool kv8_cache_ok(const void* kc, const void* vc, const void* ks, const void* vs, int64_t pages,
                  int heads, int head_dim, int block) {
  return kc != nullptr && vc != nullptr && ks != nullptr && vs != nullptr && ptr_aligned(kc, 16) &&
         ptr_aligned(vc, 16) && ptr_aligned(ks, 4) && ptr_aligned(vs, 4) && pages >= 1 &&
         pages <= INT32_MAX && heads >= 1 && heads <= 1024 && pages * heads <= INT32_MAX &&
         (head_dim == 64 || head_dim == 128) &&
         (block == 16 || block == 32 || block == 64 || block == 128);
}

bool kv8_table_ok(const void* cu, const void* lens, int64_t batch, const void* table,
                  int64_t width, int64_t ldt, const void* status) {
  return cu != nullptr && lens != nullptr && table != nullptr && ptr_aligned(cu, 4) &&
         ptr_aligned(lens, 4) && ptr_aligned(table, 4) && ptr_aligned(status, 4) && batch >= 1 &&
         batch <= 65535 && width >= 1 && width <= INT32_MAX && ldt >= width;
}

}  // namespace piq

extern "C" {
using namespace piq;

int piq_kv8_append(const void* k, const void* v, int dtype, int64_t tokens, int64_t ldk,
                   int64_t ldv, const int32_t* cu_new, const int32_t* lens_before, int64_t batch,
                   const int32_t* block_table, int64_t table_width, int64_t ldt, int8_t* k_codes,
                   int8_t* v_codes, float* k_scale, float* v_scale, int64_t pages, int kv_heads,
                   int head_dim, int block, int32_t* status, void* stream) {
  if (dtype < PIQ_BF16 || dtype > PIQ_FP32 || tokens < 0 || tokens > (int64_t)1 << 30 ||
      !kv8_cache_ok(k_codes, v_codes, k_scale, v_scale, pages, kv_heads, head_dim, block) ||
      !kv8_table_ok(cu_new, lens_before, batch, block_table, table_width, ldt, status))
    return PIQ_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(kv_heads) * head_dim;
  if (ldk < row || ldv < row || ldk % 8 != 0 || ldv % 8 != 0) return PIQ_ERR_INVALID_ARG;
  if (tokens == 0) return PIQ_OK;
  if (k == nullptr || v == nullptr || !ptr_aligned(k, 16) || !ptr_aligned(v, 16))
    return PIQ_ERR_INVALID_ARG;
  int rc = injected_fault();
  DeviceInfo info;
  if (rc == PIQ_OK) rc = device_info(&info);
  if (rc != PIQ_OK) return rc;
  Kv8Write p;
  p.k = k;
  p.v = v;
  p.tokens = tokens;
  p.ldk = ldk;
  p.ldv = ldv;
  p.cu = cu_new;
  p.lens = lens_before;
  p.table = block_table;
  p.width = table_width;
  p.ldt = ldt;
  p.kc = k_codes;
  p.vc = v_codes;
  p.ks = k_scale;
  p.vs = v_scale;
  p.pages = pages;
  p.batch = static_cast<int>(batch);
  p.heads = kv_heads;
  p.block = block;
  p.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = head_dim == 128;
  switch (dtype) {
    case PIQ_BF16:
      return wide ? launch_append<__nv_bfloat16, 128>(p, s) : launch_append<__nv_bfloat16, 64>(p, s);
    case PIQ_FP16:
      return wide ? launch_append<__half, 128>(p, s) : launch_append<__half, 64>(p, s);
    default:
      return wide ? launch_append<float, 128>(p, s) : launch_append<float, 64>(p, s);
  }
}

int piq_kv8_read(const int8_t* k_codes, const int8_t* v_codes, const float* k_scale,
                 const float* v_scale, int64_t pages, int kv_heads, int head_dim, int block,
                 const int32_t* cu_rows, const int32_t* start, int64_t batch,
                 const int32_t* block_table, int64_t table_width, int64_t ldt, int64_t rows,
                 void* k_out, void* v_out, int dtype, int64_t ldk, int64_t ldv, int32_t* status,
                 void* stream) {
  if (dtype < PIQ_BF16 || dtype > PIQ_FP32 || rows < 0 || rows > (int64_t)1 << 30 ||
      !kv8_cache_ok(k_codes, v_codes, k_scale, v_scale, pages, kv_heads, head_dim, block) ||
      !kv8_table_ok(cu_rows, start, batch, block_table, table_width, ldt, status))
    return PIQ_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(kv_heads) * head_dim;
  if (ldk < row || ldv < row || ldk % 8 != 0 || ldv % 8 != 0) return PIQ_ERR_INVALID_ARG;
  if (rows == 0) return PIQ_OK;
  if (k_out == nullptr || v_out == nullptr || !ptr_aligned(k_out, 16) || !ptr_aligned(v_out, 16))
    return PIQ_ERR_INVALID_ARG;
  int rc = injected_fault();
  DeviceInfo info;
  if (rc == PIQ_OK) rc = device_info(&info);
  if (rc != PIQ_OK) return rc;
  Kv8Read p;
  p.kc = k_codes;
  p.vc = v_codes;
  p.ks = k_scale;
  p.vs = v_scale;
  p.pages = pages;
  p.heads = kv_heads;
  p.block = block;
  p.cu = cu_rows;
  p.start = start;
  p.batch = static_cast<int>(batch);
  p.table = block_table;
  p.width = table_width;
  p.ldt = ldt;
  p.rows = rows;
  p.k = k_out;
  p.v = v_out;
  p.ldk = ldk;
  p.ldv = ldv;
  p.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = head_dim == 128;
  switch (dtype) {
    case PIQ_BF16:
      return wide ? launch_read<__nv_bfloat16, 128>(p, s) : launch_read<__nv_bfloat16, 64>(p, s);
    case PIQ_FP16:
      return wide ? launch_read<__half, 128>(p, s) : launch_read<__half, 64>(p, s);
    default:
      return wide ? launch_read<float, 128>(p, s) : launch_read<float, 64>(p, s);
  }
}

}  // extern "C"
