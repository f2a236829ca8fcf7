// Product of int8 codes on the tensor cores (tcgen05 kind::i8, int32 in TMEM):
//
//   Y[t, c] = (sum_k qx[t, k] W[c, k]) sx[t] sw[c] + bias[c]
//
// The weights are the wide operand (128 output channels a CTA, one TMEM lane
// each), the tokens the narrow one (columns), so that a few tokens cost a few
// columns and a lane of the epilogue holds one channel: a store of one token is
// 32 neighbouring channels.  Both operands are K-major tiles of 128-byte rows
// (128-byte swizzle) fetched by TMA, which fills rows past the end and the end
// of k with zeros.  Integer sums are exact, so splitting k changes nothing.
//
// Two kernels:
//  * split: one CTA a tile of 128 channels x NT tokens and a slice of k, the
//    slices of a tile in one cluster.  Few tokens read the weights once and are
//    bound by that: the k split gives every multiprocessor a part of them, and a
//    ring of 16 KB weight tiles that fills while the tokens are still being
//    quantized keeps enough bytes in flight.  The cluster adds its slices
//    through distributed shared memory, each CTA a share of the tokens.
//  * pair: persistent pairs of CTAs (cta_group::2) on tiles of 256 channels x NT
//    tokens.  Each CTA stages its 128 channels and half of the tokens: half the
//    token bytes of two lone CTAs, which is what lets shared memory keep up with
//    the tensor cores (64 B a clock written and 64 B read at NT = 256, against
//    96 and 96 alone, of 128).
//
// Warp roles: warp 0 lane 0 issues TMA, warp 1 lane 0 MMAs, the others drain
// TMEM.  Every wait is bounded; no multicast loads.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "serve.h"

namespace piq {

namespace {

constexpr int BM = 128;               // channels a CTA
constexpr int BK = 128;               // bytes of k a stage: one swizzled row
constexpr int A_TILE = BM * BK;       // 16 KB
constexpr int kRing = 192 * 1024;     // bytes of all stages
constexpr int kSmem = kRing + 1024 + 1024;  // alignment, barriers

struct GemmArgs {
  int tokens, in, out;
  int m_tiles, n_tiles;  // tiles of channels and of tokens
  int slices;            // of k (split)
  const float *sx, *sw, *bias;
  void* Y;
  int64_t ldy;
  int32_t* status;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// Instruction descriptor: kind::i8, signed A and B, s32 accumulate, K-major.
__host__ __device__ constexpr uint32_t idesc_s8(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

template <int CTAS>
__device__ __forceinline__ void umma_s8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  if constexpr (CTAS == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <typename T>
__device__ __forceinline__ void put(const GemmArgs& p, int t, int c, int acc, float sx, float sw,
                                    float bias) {
  if (t < p.tokens && c < p.out)
    static_cast<T*>(p.Y)[t * p.ldy + c] =
        from_float<T>(fmaf(static_cast<float>(acc) * sx, sw, bias));
}

// ------------------------------------------------------------------- split
template <typename T, int NT>
__global__ void __launch_bounds__(192, 1)
    int8_split_kernel(const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmX, GemmArgs p) {
  constexpr int STAGE = A_TILE + NT * BK;
  constexpr int STAGES = kRing / STAGE;
  constexpr uint32_t COLS = NT < 32 ? 32 : NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRing);
  uint64_t* empty = full + STAGES;
  uint64_t* done = empty + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slices = p.slices, slice = blockIdx.x % slices;  // a cluster is one tile's slices
  const int c0 = blockIdx.x / slices * BM, t0 = blockIdx.y * NT;
  const int num_kb = (p.in + BK - 1) / BK;
  const int kb0 = static_cast<int>(static_cast<int64_t>(num_kb) * slice / slices);
  const int kb1 = static_cast<int>(static_cast<int64_t>(num_kb) * (slice + 1) / slices);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    fence_mbar_init();
    // The weights do not depend on the kernel before this one, which lets this
    // one start only after the one before that is complete: the ring fills with
    // them while the tokens are quantized.
    const int ahead = min(STAGES, kb1 - kb0);
    for (int i = 0; i < ahead; ++i) {
      mbar_arrive_expect_tx(&full[i], STAGE);
      tma_load_2d(smem + i * STAGE, &tmW, &full[i], (kb0 + i) * BK, c0);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      for (int kb = kb0; kb < kb1; ++kb) {
        const int it = kb - kb0, st = it % STAGES;
        if (it >= STAGES) {
          if (!wait_bar(&empty[st], ((it / STAGES) & 1) ^ 1u, p.status, 61)) break;
          mbar_arrive_expect_tx(&full[st], STAGE);
          tma_load_2d(smem + st * STAGE, &tmW, &full[st], kb * BK, c0);
        }
        tma_load_2d(smem + st * STAGE + A_TILE, &tmX, &full[st], kb * BK, t0);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        const int it = kb - kb0, st = it % STAGES;
        if (!wait_bar(&full[st], (it / STAGES) & 1, p.status, 62)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(smem + st * STAGE);
        const uint64_t ad = smem_desc(a, 16, 1024, kLayoutSw128);
        const uint64_t bd = smem_desc(a + A_TILE, 16, 1024, kLayoutSw128);
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)
          umma_s8<1>(tmem, ad + 2 * kk, bd + 2 * kk, idesc_s8(BM, NT), (it | kk) != 0);
        umma_commit(&empty[st]);
      }
      if (ok) umma_commit(done);
    }
  } else {
    const int q = warp & 3;  // TMEM lanes 32 q .. : channels of the tile
    const int ch = q * 32 + lane, c = c0 + ch;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const float sw = c < p.out ? __ldg(p.sw + c) : 0.0f;
    const float bias = p.bias != nullptr && c < p.out ? __ldg(p.bias + c) : 0.0f;
    const bool ok = wait_bar(done, 0, p.status, 63);
    tc_fence_after();
    int* part = reinterpret_cast<int*>(smem);  // [NT][BM], the ring is empty now
    if (ok) {
      for (int n = 0; n < NT && t0 + n < p.tokens; n += 16) {
        float f[16];
        tmem_ld_32x32b_x16(taddr + n, f);
        if (slices == 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int t = t0 + n + i;
            put<T>(p, t, c, __float_as_int(f[i]), __ldg(p.sx + min(t, p.tokens - 1)), sw, bias);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) part[(n + i) * BM + ch] = __float_as_int(f[i]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (slices > 1) {
    cluster_sync();
    // this CTA's share of the tokens, every slice's part of them
    if (warp >= 2) {
      const int ch = (warp - 2) * 32 + lane, c = c0 + ch;
      const float sw = c < p.out ? __ldg(p.sw + c) : 0.0f;
      const float bias = p.bias != nullptr && c < p.out ? __ldg(p.bias + c) : 0.0f;
      const int live = min(NT, p.tokens - t0);
      const uint32_t base = smem_u32(smem) + 4 * ch;
      for (int n = slice; n < live; n += slices) {
        int v[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
          v[s] = s < slices ? ld_cluster(map_rank(base + 4 * BM * n, s)) : 0;
        int acc = 0;
#pragma unroll
        for (int s = 0; s < 8; ++s) acc += v[s];
        put<T>(p, t0 + n, c, acc, __ldg(p.sx + t0 + n), sw, bias);
      }
    }
    cluster_sync();  // nobody leaves while its part is read
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, COLS);
  }
}

// -------------------------------------------------------------------- pair
constexpr int kEpi = 8;  // epilogue warps a CTA: two a lane quadrant, half the columns each
constexpr int RG = 8;    // tiles of tokens a group: a wave shares few tiles of both operands

__device__ __forceinline__ void pair_tile(const GemmArgs& p, int t, int& m, int& n) {
  const int full = RG * p.m_tiles;
  const int n0 = t / full * RG;
  const int g = min(RG, p.n_tiles - n0);
  const int r = t - n0 * p.m_tiles;
  m = r / g;
  n = n0 + r - m * g;
}

// A TMA load whose bytes count on a barrier of the pair's first CTA (a cluster
// address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar,
                                                 int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
// Arrive on `bar` of both CTAs once the pair's MMAs issued so far are done.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

template <typename T, int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(64 + 32 * kEpi, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmX, GemmArgs p) {
  constexpr int STAGE = A_TILE + NT / 2 * BK;
  constexpr int STAGES = kRing / STAGE;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRing);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;  // [2]
  uint64_t* acc_empty = acc_full + 2;   // [2], the first CTA's counts both CTAs' warps
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles = p.m_tiles * p.n_tiles;
  const int num_kb = (p.in + BK - 1) / BK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpi);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(2 * NT)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full0 = map_rank(smem_u32(full), 0);
      uint32_t it = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs) {
        int m, n;
        pair_tile(p, t, m, n);
        const int c0 = (2 * m + static_cast<int>(rank)) * BM;
        const int t0 = n * NT + static_cast<int>(rank) * (NT / 2);
        for (int kb = 0; kb < num_kb; ++kb, ++it) {
          const int st = it % STAGES;
          if (!wait_bar(&empty[st], ((it / STAGES) & 1) ^ 1u, p.status, 64)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * STAGE);
          tma_load_2d_pair(smem + st * STAGE, &tmW, full0 + 8 * st, kb * BK, c0);
          tma_load_2d_pair(smem + st * STAGE + A_TILE, &tmX, full0 + 8 * st, kb * BK, t0);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      uint32_t it = 0;
      int lt = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs, ++lt) {
        const int buf = lt & 1;
        if (!wait_bar(&acc_empty[buf], ((lt >> 1) & 1) ^ 1u, p.status, 65)) break;
        tc_fence_after();
        for (int kb = 0; kb < num_kb; ++kb, ++it) {
          const int st = it % STAGES;
          if (!wait_bar(&full[st], (it / STAGES) & 1, p.status, 66)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(smem + st * STAGE);
          const uint64_t ad = smem_desc(a, 16, 1024, kLayoutSw128);
          const uint64_t bd = smem_desc(a + A_TILE, 16, 1024, kLayoutSw128);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            umma_s8<2>(tmem + buf * NT, ad + 2 * kk, bd + 2 * kk, idesc_s8(2 * BM, NT),
                       (kb | kk) != 0);
          umma_commit_pair(&empty[st]);
        }
        if (ok) umma_commit_pair(&acc_full[buf]);
      }
    }
  } else {
    const int q = warp & 3, h = (warp - 2) >> 2;
    const uint32_t free_bar = map_rank(smem_u32(acc_empty), 0);
    int lt = 0;
    for (int t = pair; t < tiles; t += pairs, ++lt) {
      int m, n;
      pair_tile(p, t, m, n);
      const int buf = lt & 1;
      const int c = (2 * m + static_cast<int>(rank)) * BM + q * 32 + lane;
      const float sw = c < p.out ? __ldg(p.sw + c) : 0.0f;
      const float bias = p.bias != nullptr && c < p.out ? __ldg(p.bias + c) : 0.0f;
      if (!wait_bar(&acc_full[buf], (lt >> 1) & 1, p.status, 67)) break;
      tc_fence_after();
      const int t0 = n * NT + h * (NT / 2);
      const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * NT + h * (NT / 2);
      for (int i0 = 0; i0 < NT / 2; i0 += 32) {
        float f[32];
        tmem_ld_32x32b_x32(taddr + i0, f);
        if (t0 + i0 + 32 <= p.tokens) {
          const float4* sx4 = reinterpret_cast<const float4*>(p.sx + t0 + i0);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 s = __ldg(sx4 + i);
            const int tt = t0 + i0 + 4 * i;
            put<T>(p, tt, c, __float_as_int(f[4 * i]), s.x, sw, bias);
            put<T>(p, tt + 1, c, __float_as_int(f[4 * i + 1]), s.y, sw, bias);
            put<T>(p, tt + 2, c, __float_as_int(f[4 * i + 2]), s.z, sw, bias);
            put<T>(p, tt + 3, c, __float_as_int(f[4 * i + 3]), s.w, sw, bias);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int tt = t0 + i0 + i;
            if (tt < p.tokens)
              put<T>(p, tt, c, __float_as_int(f[i]), __ldg(p.sx + tt), sw, bias);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(free_bar + 8 * buf);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no arrival or load of the pair is under way when a CTA leaves
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * NT)
                 : "memory");
  }
}

// -------------------------------------------------------------------- host
// [rows, cols] int8 with row stride ld as boxes of 128 bytes x box_rows.
bool code_map(CUtensorMap* map, const int8_t* q, int64_t rows, int64_t cols, int64_t ld,
              int box_rows) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t box[2] = {BK, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(q), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

typedef void (*GemmKernel)(CUtensorMap, CUtensorMap, GemmArgs);

// The shared-memory limit of each kernel, raised once on each device.
int raise_smem(GemmKernel kern, int slot) {
  static std::atomic<bool> set[64][32];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PIQ_ERR_CUDA;
  if (dev < 64 && set[dev][slot].load(std::memory_order_acquire)) return PIQ_OK;
  const int rc = cuda_rc(
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
  if (rc == PIQ_OK && dev < 64) set[dev][slot].store(true, std::memory_order_release);
  return rc;
}

int launch_gemm(GemmKernel kern, int slot, dim3 grid, int threads, int cluster,
                cudaStream_t stream, const CUtensorMap& mw, const CUtensorMap& mx,
                const GemmArgs& p) {
  const int rc = raise_smem(kern, slot);
  if (rc != PIQ_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  note_launch();
  return cuda_rc(cudaLaunchKernelEx(&cfg, kern, mw, mx, p));
}

template <typename T>
int gemm_t(const int8_t* qx, int64_t ldq, const int8_t* W, int64_t ldw, GemmArgs p,
           cudaStream_t stream, int sms) {
  static const GemmKernel split[5] = {int8_split_kernel<T, 16>, int8_split_kernel<T, 32>,
                                      int8_split_kernel<T, 64>, int8_split_kernel<T, 128>,
                                      int8_split_kernel<T, 256>};
  static const GemmKernel pair[2] = {int8_pair_kernel<T, 128>, int8_pair_kernel<T, 256>};
  const int slot0 = sizeof(T) == 4 ? 0 : std::is_same<T, __half>::value ? 8 : 16;
  const Int8Plan a = plan_int8(p.tokens, p.out, p.in, sms);
  CUtensorMap mw, mx;
  if (!code_map(&mw, W, p.out, p.in, ldw, BM) ||
      !code_map(&mx, qx, p.tokens, p.in, ldq, a.pair ? a.nt / 2 : a.nt))
    return PIQ_ERR_INVALID_ARG;
  p.n_tiles = static_cast<int>(ceil_div(p.tokens, a.nt));
  if (a.pair) {
    p.m_tiles = static_cast<int>(ceil_div(p.out, 2 * BM));
    const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
    if (tiles > INT32_MAX) return PIQ_ERR_INVALID_ARG;
    const int pairs = static_cast<int>(std::min<int64_t>(tiles, sms / 2));
    const int i = a.nt == 256;
    return launch_gemm(pair[i], slot0 + i, dim3(2 * pairs), 64 + 32 * kEpi, 0, stream, mw, mx, p);
  }
  p.m_tiles = static_cast<int>(ceil_div(p.out, BM));
  p.slices = a.slices;
  int i = 0;
  while (16 << i < a.nt) ++i;
  return launch_gemm(split[i], slot0 + 2 + i, dim3(a.slices * p.m_tiles, p.n_tiles), 192, a.slices,
                     stream, mw, mx, p);
}

}  // namespace

EncodeTiledFn tensor_map_encoder() {
  static const EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &qr) !=
            cudaSuccess ||
        qr != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<EncodeTiledFn>(ptr);
  }();
  return fn;
}

// Tiles of one product.  Many tokens: pairs, on 256-token tiles when those give
// every pair of multiprocessors work, else on 128-token tiles while they do.
// Fewer: single CTAs, the widest token tile that still gives most multiprocessors a
// tile, and k cut into up to eight slices (each at least four 128-byte steps)
// when the tiles alone do not.
Int8Plan plan_int8(int64_t tokens, int64_t out, int64_t in, int sms) {
  Int8Plan a;
  const int64_t mp = ceil_div(out, 2 * BM), m1 = ceil_div(out, BM);
  a.pair = true;
  a.slices = 1;
  a.nt = 256;
  if (tokens > 128 && mp * ceil_div(tokens, 256) >= sms / 2) return a;
  a.nt = 128;
  if (tokens > 128 && mp * ceil_div(tokens, 128) >= sms / 2 * 3 / 4) return a;
  a.pair = false;
  a.nt = 256;
  while (a.nt > 16 && (ceil_div(tokens, a.nt / 2) == 1 ||
                       (a.nt > 64 && m1 * ceil_div(tokens, a.nt) < sms * 3 / 4)))
    a.nt /= 2;
  const int64_t tiles = m1 * ceil_div(tokens, a.nt), kb = ceil_div(in, BK);
  while (a.slices < 8 && tiles * a.slices * 2 <= sms && kb >= 8 * a.slices) a.slices *= 2;
  return a;
}

int launch_int8_gemm(const int8_t* qx, int64_t ldq, const float* sx, int64_t tokens, int64_t in,
                     const int8_t* W, int64_t out, int64_t ldw, const float* sw, const float* bias,
                     void* Y, int dtype, int64_t ldy, int32_t* status, cudaStream_t stream) {
  DeviceInfo info;
  const int rc = device_info(&info);
  if (rc != PIQ_OK) return rc;
  GemmArgs p{};
  p.tokens = static_cast<int>(tokens);
  p.in = static_cast<int>(in);
  p.out = static_cast<int>(out);
  p.sx = sx;
  p.sw = sw;
  p.bias = bias;
  p.Y = Y;
  p.ldy = ldy;
  p.status = status;
  switch (dtype) {
    case PIQ_BF16: return gemm_t<__nv_bfloat16>(qx, ldq, W, ldw, p, stream, info.sm_count);
    case PIQ_FP16: return gemm_t<__half>(qx, ldq, W, ldw, p, stream, info.sm_count);
    default: return gemm_t<float>(qx, ldq, W, ldw, p, stream, info.sm_count);
  }
}

}  // namespace piq
