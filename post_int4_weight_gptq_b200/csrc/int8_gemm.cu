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
constexpr int kSmallRing = 96 * 1024; // of the split kernel on up to 64 tokens: two CTAs share
                                      // a multiprocessor, one starting while the other ends
constexpr int kSmemExtra = 1024 + 1024;  // alignment, barriers
constexpr int split_ring(int nt) { return nt <= 64 ? kSmallRing : kRing; }

struct GemmArgs {
  int tokens, in, out;
  int m_tiles, n_tiles;  // tiles of channels and of tokens
  int slices;            // of k (split)
  const float *sx, *sw, *bias;
  void* Y;
  int64_t ldy;
  bool wide;  // Y and its rows are 16-byte aligned
  int32_t* status;
  uint64_t wait_ns;  // limit of a wait
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
__device__ __forceinline__ int4 ld_cluster(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_cluster_word(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
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

__device__ __forceinline__ float scaled(int acc, float sx, float sw, float bias) {
  return fmaf(static_cast<float>(acc) * sx, sw, bias);
}

// N tokens (t0 ..) of a warp's 32 channels (c0 .., one a lane, accumulators in f) to
// Y through the warp's staging rows: a lane holds a channel of every token, a store
// wants neighbouring channels of one.  Stores of one channel a lane took the tile of
// 256 tokens 6 us; this takes an eighth of their instructions.
template <typename T, int N>
__device__ __forceinline__ void store_tokens(const GemmArgs& p, T* stage, const float (&f)[N],
                                             const float4* sx4, int t0, int c0, float sw,
                                             float bias, int lane) {
  constexpr int PER = 16 / sizeof(T), PIECES = 32 / PER;  // channels a piece, pieces a token
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const float4 s = sx4[i];
    stage[(4 * i) * 32 + lane] = from_float<T>(scaled(__float_as_int(f[4 * i]), s.x, sw, bias));
    stage[(4 * i + 1) * 32 + lane] =
        from_float<T>(scaled(__float_as_int(f[4 * i + 1]), s.y, sw, bias));
    stage[(4 * i + 2) * 32 + lane] =
        from_float<T>(scaled(__float_as_int(f[4 * i + 2]), s.z, sw, bias));
    stage[(4 * i + 3) * 32 + lane] =
        from_float<T>(scaled(__float_as_int(f[4 * i + 3]), s.w, sw, bias));
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < N * PIECES / 32; ++i) {
    const int piece = i * 32 + lane, t = t0 + piece / PIECES, c = c0 + piece % PIECES * PER;
    const uint4 v = reinterpret_cast<const uint4*>(stage)[piece];
    T* y = static_cast<T*>(p.Y) + t * p.ldy + c;
    if (t < p.tokens) {
      if (p.wide && c + PER <= p.out) {
        *reinterpret_cast<uint4*>(y) = v;
      } else {
        const T* e = stage + piece * PER;
        for (int j = 0; j < PER && c + j < p.out; ++j) y[j] = e[j];
      }
    }
  }
  __syncwarp();
}

// NaN for tokens [t0, t0 + n) of channel c, behind a wait that gave up.
template <typename T>
__device__ __forceinline__ void store_nan(const GemmArgs& p, int t0, int n, int c) {
  if (c >= p.out) return;
  for (int t = t0; t < min(t0 + n, p.tokens); ++t)
    static_cast<T*>(p.Y)[t * p.ldy + c] = from_float<T>(__uint_as_float(0x7FC00000u));
}

// ------------------------------------------------------------------- split
template <typename T, int NT>
__global__ void __launch_bounds__(192, NT <= 64 ? 2 : 1)
    int8_split_kernel(const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmX, GemmArgs p) {
  constexpr int RING = split_ring(NT);
  constexpr int STAGE = A_TILE + NT * BK;
  constexpr int STAGES = RING / STAGE;
  constexpr uint32_t COLS = NT < 32 ? 32 : NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + RING);
  uint64_t* empty = full + STAGES;
  uint64_t* done = empty + STAGES;
  uint64_t* drain = done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  __shared__ __align__(16) float s_sx[NT];
  __shared__ uint32_t s_bad;  // a wait of this CTA gave up
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
    mbar_init(drain, 1);
    s_bad = 0;
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

  int copies = 0;      // steps whose copies the copying thread has asked for
  bool began = false;  // the issuing thread has issued products
  if (warp == 0) {
    if (lane == 0) {
      for (int kb = kb0; kb < kb1; ++kb, ++copies) {
        const int it = kb - kb0, st = it % STAGES;
        if (it >= STAGES) {
          if (!wait_bar(&empty[st], ((it / STAGES) & 1) ^ 1u, p.wait_ns, p.status, 61)) {
            s_bad = 1;
            break;
          }
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
        if (!wait_bar(&full[st], (it / STAGES) & 1, p.wait_ns, p.status, 62)) {
          ok = false;
          s_bad = 1;
          break;
        }
        began = true;
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
    // the tokens' scales, for all four warps
    for (int i = threadIdx.x - 64; i < NT; i += 128)
      s_sx[i] = __ldg(p.sx + min(t0 + i, p.tokens - 1));
    asm volatile("bar.sync 1, 128;" ::: "memory");
    const bool ok = wait_warp(done, 0, p.wait_ns, p.status, 63);
    tc_fence_after();
    // the ring is empty now: staging of the stores, or this slice's sums [NT][BM]
    constexpr int CH = NT < 32 ? NT : 32;
    T* const stage = reinterpret_cast<T*>(smem) + q * (CH * 32);
    int* const part = reinterpret_cast<int*>(smem);
    if (ok) {
      for (int n = 0; n < NT && t0 + n < p.tokens; n += CH) {
        float f[CH];
        if constexpr (CH == 32)
          tmem_ld_32x32b_x32(taddr + n, f);
        else
          tmem_ld_32x32b_x16(taddr + n, f);
        if (slices == 1) {
          store_tokens<T, CH>(p, stage, f, reinterpret_cast<const float4*>(s_sx + n), t0 + n,
                              c0 + q * 32, sw, bias, lane);
        } else {
#pragma unroll
          for (int i = 0; i < CH; ++i) part[(n + i) * BM + ch] = __float_as_int(f[i]);
        }
      }
    } else {
      s_bad = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (s_bad) {
    // what is under way ends before anyone reads the ring or leaves: the last copies into
    // every stage (of each step both tiles were asked for), and the products
    if (warp == 0 && lane == 0) {
      const uint64_t now = global_timer_ns();
      for (int it = max(copies - STAGES, 0); it < copies; ++it)
        drain_bar(&full[it % STAGES], (it / STAGES) & 1, now);
    } else if (warp == 1 && lane == 0 && began) {
      umma_commit(drain);
      drain_bar(drain, 0, global_timer_ns());
    }
    __syncthreads();
  }
  if (slices > 1) {
    cluster_sync();
    // this CTA's share of the tokens: a warp a token, four channels a lane, every
    // slice's sums read at once
    if (warp >= 2) {
      const int c = c0 + 4 * lane;
      float sw[4], bias[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sw[j] = c + j < p.out ? __ldg(p.sw + c + j) : 0.0f;
        bias[j] = p.bias != nullptr && c + j < p.out ? __ldg(p.bias + c + j) : 0.0f;
      }
      const int live = min(NT, p.tokens - t0);
      const uint32_t base = smem_u32(smem) + 16 * lane;
#pragma unroll 2
      for (int n = slice + slices * (warp - 2); n < live; n += 4 * slices) {
        int4 v[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
          v[s] = s < slices ? ld_cluster(map_rank(base + 4 * BM * n, s)) : make_int4(0, 0, 0, 0);
        int4 a = v[0];
#pragma unroll
        for (int s = 1; s < 8; ++s) {
          a.x += v[s].x;
          a.y += v[s].y;
          a.z += v[s].z;
          a.w += v[s].w;
        }
        const float sx = s_sx[n];
        T y[4] = {from_float<T>(scaled(a.x, sx, sw[0], bias[0])),
                  from_float<T>(scaled(a.y, sx, sw[1], bias[1])),
                  from_float<T>(scaled(a.z, sx, sw[2], bias[2])),
                  from_float<T>(scaled(a.w, sx, sw[3], bias[3]))};
        T* to = static_cast<T*>(p.Y) + (t0 + n) * p.ldy + c;
        if (p.wide && c + 4 <= p.out) {
          if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float4*>(to) = make_float4(y[0], y[1], y[2], y[3]);
          else
            *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(y);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c + j < p.out) to[j] = y[j];
        }
      }
    }
    cluster_sync();  // nobody leaves while its part is read
  }
  // this slice is missing in what the cluster has stored
  if (s_bad && warp >= 2) store_nan<T>(p, t0, NT, c0 + (warp & 3) * 32 + lane);
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

// The same on this CTA's `bar` alone.
__device__ __forceinline__ void umma_commit_pair_here(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}
// `bytes` that no copy will bring are taken off the current phase of `bar`.
__device__ __forceinline__ void mbar_forgo_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(
                   smem_u32(bar)),
               "r"(bytes)
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
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  __shared__ uint32_t s_bad;        // a wait of either CTA gave up
  __shared__ uint32_t s_copies[2];  // steps whose copies each CTA has asked for
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
    mbar_init(drain, 1);
    s_bad = 0;
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
  auto gave_up = [&]() {  // both CTAs know it behind the barrier at the end
    for (uint32_t r = 0; r < 2; ++r) st_cluster_word(map_rank(smem_u32(&s_bad), r), 1);
  };

  bool began = false;  // the issuing thread has issued products
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
          if (!wait_bar(&empty[st], ((it / STAGES) & 1) ^ 1u, p.wait_ns, p.status, 64)) {
            ok = false;
            gave_up();
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * STAGE);
          tma_load_2d_pair(smem + st * STAGE, &tmW, full0 + 8 * st, kb * BK, c0);
          tma_load_2d_pair(smem + st * STAGE + A_TILE, &tmX, full0 + 8 * st, kb * BK, t0);
        }
      }
      for (uint32_t r = 0; r < 2; ++r) st_cluster_word(map_rank(smem_u32(&s_copies[rank]), r), it);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      uint32_t it = 0;
      int lt = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs, ++lt) {
        const int buf = lt & 1;
        if (!wait_bar(&acc_empty[buf], ((lt >> 1) & 1) ^ 1u, p.wait_ns, p.status, 65)) {
          gave_up();
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < num_kb; ++kb, ++it) {
          const int st = it % STAGES;
          if (!wait_bar(&full[st], (it / STAGES) & 1, p.wait_ns, p.status, 66)) {
            ok = false;
            gave_up();
            break;
          }
          began = true;
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
    T* const stage = reinterpret_cast<T*>(smem + kRing + 1024) + (warp - 2) * (32 * 32);
    int lt = 0;
    bool ok = true;
    for (int t = pair; t < tiles; t += pairs, ++lt) {
      int m, n;
      pair_tile(p, t, m, n);
      const int buf = lt & 1;
      const int c = (2 * m + static_cast<int>(rank)) * BM + q * 32 + lane;
      const float sw = c < p.out ? __ldg(p.sw + c) : 0.0f;
      const float bias = p.bias != nullptr && c < p.out ? __ldg(p.bias + c) : 0.0f;
      const int t0 = n * NT + h * (NT / 2);
      if (ok && !wait_warp(&acc_full[buf], (lt >> 1) & 1, p.wait_ns, p.status, 67)) {
        ok = false;
        if (lane == 0) gave_up();
      }
      if (!ok) {  // this tile and those after it
        store_nan<T>(p, t0, NT / 2, c);
        continue;
      }
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * NT + h * (NT / 2);
      for (int i0 = 0; i0 < NT / 2 && t0 + i0 < p.tokens; i0 += 32) {
        float f[32];
        tmem_ld_32x32b_x32(taddr + i0, f);
        float4 sx[8];
        if (t0 + i0 + 32 <= p.tokens) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            sx[i] = __ldg(reinterpret_cast<const float4*>(p.sx + t0 + i0) + i);
        } else {
          const int last = p.tokens - 1, at = t0 + i0;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            sx[i] = make_float4(__ldg(p.sx + min(at + 4 * i, last)),
                                __ldg(p.sx + min(at + 4 * i + 1, last)),
                                __ldg(p.sx + min(at + 4 * i + 2, last)),
                                __ldg(p.sx + min(at + 4 * i + 3, last)));
        }
        store_tokens<T, 32>(p, stage, f, sx, t0 + i0, c - lane, sw, bias, lane);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(free_bar + 8 * buf);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no arrival or load of the pair is under way when a CTA leaves
  if (s_bad) {  // in both CTAs
    // After a wait that gave up some are.  The first CTA holds the barriers: it waits for
    // its products, and for the last copies of both into every stage, where one may have
    // gone a few steps further than the other.
    if (rank == 0 && warp == 1 && lane == 0 && began) {
      umma_commit_pair_here(drain);
      drain_bar(drain, 0, global_timer_ns());
    } else if (rank == 0 && warp == 0 && lane == 0) {
      const uint64_t now = global_timer_ns();
      const int mine = s_copies[0], other = s_copies[1], all = max(mine, other);
      for (int it = max(all - STAGES, 0); it < all; ++it) {
        uint64_t* const bar = &full[it % STAGES];
        if (it >= mine)
          mbar_arrive_expect_tx(bar, STAGE);  // only the other's
        else if (it >= other)
          mbar_forgo_tx(bar, STAGE);          // only this one's
        drain_bar(bar, (it / STAGES) & 1, now);
      }
    }
    __syncthreads();
    cluster_sync();
  }
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
int raise_smem(GemmKernel kern, int slot, int smem) {
  static std::atomic<bool> set[64][32];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PIQ_ERR_CUDA;
  if (dev < 64 && set[dev][slot].load(std::memory_order_acquire)) return PIQ_OK;
  const int rc = cuda_rc(
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  if (rc == PIQ_OK && dev < 64) set[dev][slot].store(true, std::memory_order_release);
  return rc;
}

int launch_gemm(GemmKernel kern, int slot, dim3 grid, int threads, int ring, int cluster,
                cudaStream_t stream, const CUtensorMap& mw, const CUtensorMap& mx,
                const GemmArgs& p) {
  const int smem = ring + kSmemExtra;
  const int rc = raise_smem(kern, slot, smem);
  if (rc != PIQ_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
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
    if (tiles > INT32_MAX - sms) return PIQ_ERR_INVALID_ARG;
    const int pairs = static_cast<int>(std::min<int64_t>(tiles, sms / 2));
    const int i = a.nt == 256;
    return launch_gemm(pair[i], slot0 + i, dim3(2 * pairs), 64 + 32 * kEpi,
                       kRing + kEpi * 32 * 32 * static_cast<int>(sizeof(T)), 0, stream, mw, mx, p);
  }
  p.m_tiles = static_cast<int>(ceil_div(p.out, BM));
  p.slices = a.slices;
  int i = 0;
  while (16 << i < a.nt) ++i;
  return launch_gemm(split[i], slot0 + 2 + i, dim3(a.slices * p.m_tiles, p.n_tiles), 192,
                     split_ring(a.nt), a.slices, stream, mw, mx, p);
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

// Tiles of one product.  The forms differ in the tiles that run at once and in the
// time of one tile (relative, measured at in = 4096: 256 x 256 on a pair 4.0, 256 x
// 128 3.0, 128 x 256 on one CTA 4.2, 128 x 128 3.1, 128 x 64 with two CTAs a
// multiprocessor 2.9); the one with the least waves times time is taken.  1024 x 4096
// -> 4096 took 20.6 us on pairs of 256, 26.0 on pairs of 128, 29.2 on 64; 512 tokens
// 19.4, 17.0 and 15.6.  Up to 64 tokens fit one tile, as narrow as they are.  Where
// the tiles leave multiprocessors idle, k is cut into up to eight slices of at least
// eight 128-byte steps (37 x 11008 -> 4096: 29 us whole, 14 us in eight; 64 x 4096 ->
// 11008, 86 tiles, gains nothing from two and loses with four).
Int8Plan plan_int8(int64_t tokens, int64_t out, int64_t in, int sms) {
  Int8Plan a;
  a.pair = false;
  a.slices = 1;
  a.nt = 64;
  const int64_t m1 = ceil_div(out, BM), m2 = ceil_div(out, 2 * BM);
  if (tokens > 64) {
    struct Form {
      bool pair;
      int nt, at_once, time;
    };
    const Form forms[] = {{false, 64, 2 * sms, 29},
                          {false, 128, sms, 31},
                          {true, 128, sms / 2, 30},
                          {true, 256, sms / 2, 40},
                          {false, 256, sms, 42}};
    int64_t best = INT64_MAX;
    for (const Form& f : forms) {
      const int64_t tiles = (f.pair ? m2 : m1) * ceil_div(tokens, f.nt);
      const int64_t t = ceil_div(tiles, f.at_once) * f.time;
      // (the grid's second dimension holds the split kernel's token tiles)
      if (t < best && (f.pair || ceil_div(tokens, f.nt) <= 65535)) {
        best = t;
        a.pair = f.pair;
        a.nt = f.nt;
      }
    }
  } else {
    while (a.nt > 16 && tokens <= a.nt / 2) a.nt /= 2;
  }
  if (!a.pair) {
    const int64_t tiles = m1 * ceil_div(tokens, a.nt), kb = ceil_div(in, BK);
    const int64_t room = a.nt <= 64 ? 2 * sms : sms;
    while (a.slices < 8 && tiles * a.slices * 2 <= room && kb >= 16 * a.slices) a.slices *= 2;
  }
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
  const int size = dtype == PIQ_FP32 ? 4 : 2;
  p.wide = ptr_aligned(Y, 16) && ldy * size % 16 == 0;
  p.status = status;
  p.wait_ns = serving_wait_ns();
  switch (dtype) {
    case PIQ_BF16: return gemm_t<__nv_bfloat16>(qx, ldq, W, ldw, p, stream, info.sm_count);
    case PIQ_FP16: return gemm_t<__half>(qx, ldq, W, ldw, p, stream, info.sm_count);
    default: return gemm_t<float>(qx, ldq, W, ldw, p, stream, info.sm_count);
  }
}

}  // namespace piq
