// Attention of new tokens over the 8-bit paged cache, a chunk of keys at a time.
//
//   x_j = scale q . (k_scale k_j),  out = sum_j 2^(x_j') v_scale v_j / sum_j 2^(x_j')
//
// (x' = x log2 e - running maximum).  Every warp has a ring of its own in shared
// memory, filled by TMA with tiles of 32 keys and values (a copy is issued when the
// warp has read the stage before; copies into registers kept too few bytes under
// way, and cp.async of scattered 16-byte pieces took 20 cycles of the shared-memory
// pipe an instruction).  From there 16-byte reads give matrix fragments as they
// are, because the order of the dimensions inside a fragment is free as long as q's
// agrees: lane (r, c) = (lane / 4, lane % 4) takes bytes 16 c .. of a token for the
// scores, and one eighth of the dimensions of four tokens for the values.  The
// tokens' places in a tile of 16 and the eighths are permuted so that the swizzled
// reads of eight lanes meet 32 different banks.
//
// A byte becomes a half exactly: u = code + 128 under the exponent of 1024 is 1152 +
// code, minus 1152.  (Leaving the 128 in and taking it off the sums instead was no
// faster, 54.6 against 54.4 us for one sequence of 131072 keys, and its cancellation
// put lse off by 5e-5 where a query has a few loud channels; this way 2e-6.)
//
// Keys and values are the wide operand (16 tokens, or 16 dimensions, a
// product), the queries the narrow one (8 rows), because a decoding step has
// few rows for every key: S^T = K q^T and O^T = V^T P^T, with P^T's fragment
// made from S^T's by an 8x8 transpose in registers.
//
// Probabilities enter the second product in fp16 as 2^7 p v_scale / (largest
// v_scale that the row has seen, as a power of two), p relative to a running maximum
// that moves only when a score exceeds it by 2^7: below 2^15, and what is more than
// 2^31 below the largest is lost.  The sum of p stays in fp32.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "kv8_attn.cuh"

namespace piq {

namespace {

constexpr int kWarps = 6;
// Bytes of a warp's ring: two stages of 32 keys and values.
constexpr int ring_bytes(int dim) { return 2 * 64 * dim; }
// CTAs that share a multiprocessor, as their registers allow (three of 64 dimensions
// and one group of rows instead of two: 67.9 -> 64.1 us on 48 ragged sequences).
constexpr int ctas_sm(int dim, int nt) { return (dim == 64 ? 4 : 3) - nt; }
constexpr int kMaxPages = 256;        // pages of a chunk (4096 keys, blocks of 16)

// Bytes 0 and 2, and 1 and 3, of four codes, as halves (low = 0x00FF00FF).
__device__ __forceinline__ void halves_of(uint32_t w, uint32_t low, uint32_t& even, uint32_t& odd) {
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const uint32_t e = (w & low) ^ 0x64806480u;
  const uint32_t o = ((w >> 8) & low) ^ 0x64806480u;
  const __half2 eh = __hsub2(*reinterpret_cast<const __half2*>(&e), off);
  const __half2 oh = __hsub2(*reinterpret_cast<const __half2*>(&o), off);
  even = *reinterpret_cast<const uint32_t*>(&eh);
  odd = *reinterpret_cast<const uint32_t*>(&oh);
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The token that row k of a tile of 16 stands for (k < 8; the others are 8 further
// on).  Rows of 128 bytes (128-byte swizzle): k and k + 1 are four apart, so that
// their halves of a row lie in other banks.  Rows of 64 (64-byte swizzle, two a
// line): k and k + 1 lie in other halves of a line, and of the even ones (and the
// odd ones) two in either half, in lines two apart.
template <int D>
__device__ __forceinline__ int token_of(int k) {
  const int c = k >> 1, odd = k & 1;
  return D == 128 ? odd * 4 + c : ((c >> 1) * 4 + (c & 1)) ^ (odd * 3);
}

// NT groups of eight query rows of one kv head (rows are (token, head) pairs,
// the heads of the group fastest) against one chunk of keys.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, ctas_sm(D, NT)) kv8_chunk_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, Kv8Attn p) {
  constexpr int ROWS = 8 * NT;
  constexpr int KS = D / 16;   // k steps of the scores = 16-row tiles of the output
  constexpr int KV = D / 64;   // 16-byte loads of a key a lane; value loads are 4 of D / 8 bytes
  constexpr int STAGE = 64 * D;            // bytes of 32 keys, then their 32 values
  constexpr int kRing = ring_bytes(D), STAGES = kRing / STAGE;
  __shared__ int s_page[kMaxPages];  // page kv_heads + head
  __shared__ float s_ks[kMaxPages], s_vs[kMaxPages];
  __shared__ __align__(16) __half s_q[ROWS][D];
  __shared__ float s_rs[ROWS];
  __shared__ float s_m[kWarps][ROWS], s_l[kWarps][ROWS], s_d[kWarps][ROWS];
  __shared__ uint64_t full[kWarps][STAGES];
  extern __shared__ uint8_t ring_raw[];  // the warps' rings, then the join's buffer
  uint8_t* const ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(ring_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* const s_o = reinterpret_cast<float*>(ring);
  static_assert(sizeof(float) * NT * KS * 4 * 32 <= kRing, "join buffer");

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane < STAGES) mbar_init(&full[warp][lane], 1);
  fence_mbar_init();
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait();
  const int r = lane >> 2, c = lane & 3;
  const int b = blockIdx.z;
  const int row_groups = static_cast<int>(gridDim.x) / p.kv_heads;
  const int kvh = blockIdx.x / row_groups, rg = blockIdx.x % row_groups;
  const int part = blockIdx.y;
  const int64_t q0 = __ldg(p.cu + b), q1 = __ldg(p.cu + b + 1), seq_len = __ldg(p.lens + b);
  if (q0 == q1) return;
  T* out = static_cast<T*>(p.out);
  if (bad_lengths(p, q0, q1, seq_len)) {
    if (blockIdx.x == 0 && part == 0) report_lengths<T, D>(p, b, q0, q1);
    return;
  }
  const int n = static_cast<int>(q1 - q0), len = static_cast<int>(seq_len);
  const int rows = n * p.group;
  const int row0 = rg * ROWS;
  if (row0 >= rows) return;
  const int origin = first_block_key(len, n, p.window, p.block);
  const int k0 = origin + part * p.chunk;
  if (k0 >= len) return;
  const int nkeys = min(p.chunk, len - k0);
  const bool single = len - origin <= p.chunk;  // this CTA has all the sequence's keys
  const int shift = __ffs(p.block) - 1;

  // -------------------------------------------------- pages and scales, queries
  // The rows' values are asked for first, the page table's entries and their scales
  // next: the waits overlap.
  constexpr int QW = (ROWS + kWarps - 1) / kWarps;  // rows a warp
  float qv[QW][D / 32];
#pragma unroll
  for (int i = 0; i < QW; ++i) {
    const int at = min(warp + i * kWarps, ROWS - 1);  // the last row may come twice
    const unsigned row = row0 + at;
    const unsigned tok = row / p.group, head = row - tok * p.group;
    const T* src = static_cast<const T*>(p.q) + (q0 + tok) * p.ldq + (kvh * p.group + head) * D;
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
      qv[i][j] = row < static_cast<unsigned>(rows) ? to_float(__ldg(src + 32 * j + lane)) : 0.0f;
  }
  // ------------------------------------------------------------- the keys, 32 a step
  // Two tiles of 16 keys: two independent chains of products, and the votes and
  // address work once for both.
  const int ntiles = (nkeys + 15) / 16;
  const int steps = (nkeys + 31) / 32;
  const int tshift = shift - 4;  // log2 of the tiles of a page
  const int in_page = (1 << tshift) - 1;
  uint8_t* const mine = ring + warp * kRing;
  auto fetch = [&](int step, int stage, auto page_of) {  // lane 0; page_of(i): place of page i
    uint8_t* to = mine + stage * STAGE;
    const int tile = 2 * step;
    if (tshift > 0) {  // 32 keys of one page (those past the last one lie in it too)
      mbar_arrive_expect_tx(&full[warp][stage], STAGE);
      const int z = page_of(tile >> tshift), y = (tile & in_page) * 16;
      tma_load_3d(to, &tm_k, &full[warp][stage], 0, y, z);
      tma_load_3d(to + 32 * D, &tm_v, &full[warp][stage], 0, y, z);
    } else {           // pages of 16
      const int two = tile + 1 < ntiles ? 2 : 1;
      mbar_arrive_expect_tx(&full[warp][stage], two * (STAGE / 2));
      for (int u = 0; u < two; ++u) {
        const int z = page_of(tile + u);
        tma_load_3d(to + u * (16 * D), &tm_k, &full[warp][stage], 0, 0, z);
        tma_load_3d(to + 32 * D + u * (16 * D), &tm_v, &full[warp][stage], 0, 0, z);
      }
    }
  };
  // The first stages go out before anything else is known but the pages.
  const int npages = (nkeys + p.block - 1) >> shift;
  const int32_t* table = p.table + b * p.ldt + (k0 >> shift);
  if (lane == 0) {
    auto direct = [&](int i) {
      const int pg = __ldg(table + i);
      return (pg >= 0 && pg < p.pages ? pg : 0) * p.kv_heads + kvh;
    };
#pragma unroll 1
    for (int i = 0; i < STAGES; ++i)
      if (warp + i * kWarps < steps) fetch(warp + i * kWarps, i, direct);
  }
  __syncwarp();
  for (int i = threadIdx.x; i < npages; i += blockDim.x) {
    int pg = __ldg(table + i);
    float ks = __uint_as_float(0x7FC00000u), vs = ks;
    if (pg >= 0 && pg < p.pages) {
      ks = __ldg(p.ks + static_cast<int64_t>(pg) * p.kv_heads + kvh);
      vs = __ldg(p.vs + static_cast<int64_t>(pg) * p.kv_heads + kvh);
    } else {
      note_status(p.status, PIQ_ERR_INVALID_ARG, b);
      pg = 0;
    }
    s_page[i] = pg * p.kv_heads + kvh;
    s_ks[i] = ks;
    s_vs[i] = vs;
  }
#pragma unroll
  for (int i = 0; i < QW; ++i) {
    float amax = 0.0f;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      amax = fmaxf(amax, fabsf(qv[i][j]));
      nan |= !(qv[i][j] == qv[i][j]);
    }
    amax = warp_max(amax);
    if (__any_sync(0xffffffffu, nan)) amax = __uint_as_float(0x7FC00000u);
    float mul;
    const float undo = row_exponent<T>(amax, mul);
    const int at = min(warp + i * kWarps, ROWS - 1);
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
      s_q[at][32 * j + lane] = __float2half_rn(undo == undo ? qv[i][j] * mul : 0.0f);
    if (lane == 0) s_rs[at] = undo * p.scale2;
  }
  __syncthreads();

  // where this lane's pieces lie in a swizzled tile of 16 tokens
  const int tk = token_of<D>(r);
  const int k_at = D == 128 ? tk * 128 + ((c ^ tk) << 4) : tk * 64 + ((c ^ (tk >> 1)) << 4);
  const int eighth = D == 128 ? (r & 1) * 4 + (r >> 1) : r;  // dimensions eighth D / 8 ..
  int v_at[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int tv = token_of<D>(2 * c + h);
    v_at[h] = 32 * D + (D == 128 ? tv * 128 + ((eighth ^ tv) << 4)
                                 : tv * 64 + (((r >> 1) ^ (tv >> 1)) << 4) + (r & 1) * 8);
  }

  // -------------------------------------------------------------- fragments of q
  uint32_t qf[NT][KS][2];
  float rs[NT][2];
  int hi[NT][2];  // keys of the chunk that rows 2c, 2c + 1 see: j < hi
  const int window = p.window;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      // bytes 16 c + 4 w + {0, 2} and {1, 3} of each 64-byte half, w = s % 4
      const uint2 x = *reinterpret_cast<const uint2*>(
          &s_q[8 * t + r][64 * (s / 4) + 16 * c + 4 * (s % 4)]);
      qf[t][s][0] = __byte_perm(x.x, x.y, 0x5410);
      qf[t][s][1] = __byte_perm(x.x, x.y, 0x7632);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = row0 + 8 * t + 2 * c + e;
      rs[t][e] = s_rs[8 * t + 2 * c + e];
      const int tok = static_cast<int>(static_cast<unsigned>(row) / p.group);
      hi[t][e] = row < rows ? len - n + tok + 1 - k0 : 0;
    }
  }
  // Tiles in which every row sees every key need no masks.  (Rows that do not exist see
  // none, so that a group of fewer than eight rows masks every step.)
  const unsigned last_tok = static_cast<unsigned>(min(row0 + ROWS, rows) - 1) / p.group;
  const unsigned first_tok = static_cast<unsigned>(row0) / p.group;
  const int all_lo =
      window > 0 ? max(len - n + static_cast<int>(last_tok) + 1 - window - k0, 0) : 0;
  const int all_hi = row0 + ROWS <= rows ? len - n + static_cast<int>(first_tok) + 1 - k0 : 0;

  float m[NT][2], l[NT][2], vc[NT][2], o[NT][KS][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t][0] = m[t][1] = kLow;
    l[t][0] = l[t][1] = 0.0f;
    vc[t][0] = vc[t][1] = kFirstFactor;
#pragma unroll
    for (int j = 0; j < KS; ++j) o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.0f;
  }

  int stage = 0;
  const uint32_t mine_at = smem_u32(mine), low = p.low_bytes;
  uint32_t phase = 0;
  bool ok = true;
  // One step; MASK: some row does not see all of its keys.  Two forms, because the
  // compiler would turn a branch around the masks into selects on every step.
  auto process = [&](int step, auto mask_c) {
    constexpr bool MASK = decltype(mask_c)::value;
    const uint32_t at = mine_at + stage * STAGE;
    const int key0 = 32 * step;
    float s[2][NT][4] = {}, kscale[2], vscale[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // a second tile behind the last keys is all masked; it borrows a page's scales
      const int page = (MASK ? min(2 * step + u, ntiles - 1) : 2 * step + u) >> tshift;
      kscale[u] = s_ks[page];
      vscale[u] = s_vs[page];
    }
#pragma unroll
    for (int j = 0; j < KV; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint4 w0 = lds128(at + (k_at ^ (64 * j)) + u * (16 * D));
        const uint4 w1 = lds128(at + (k_at ^ (64 * j)) + u * (16 * D) + 8 * D);
        const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0, a1, a2, a3;
          halves_of(x0[w], low, a0, a2);
          halves_of(x1[w], low, a1, a3);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma_f16(s[u][t], a0, a1, a2, a3, qf[t][4 * j + w][0], qf[t][4 * j + w][1]);
        }
      }

    // scores in log2 units
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float f0 = rs[t][0] * kscale[u], f1 = rs[t][1] * kscale[u];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[u][t][e] *= e & 1 ? f1 : f0;
          if (MASK) {
            const int j = key0 + 16 * u + tk + 8 * (e >> 1), h = hi[t][e & 1];
            const bool see = j < h && (window == 0 || j >= h - window);
            if (!see) s[u][t][e] = __uint_as_float(0xFF800000u);
          }
        }
      }
    bool over = false;
    const float vs_top = fmaxf(fmaxf(vscale[0], vscale[1]), 0.0f);  // (not NaN)
    float top[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[t][e] = fmaxf(fmaxf(s[0][t][e], s[0][t][e + 2]), fmaxf(s[1][t][e], s[1][t][e + 2]));
        // (a masked row that sees none of the keys, or is none, has no say)
        over |= top[t][e] > m[t][e] + kSlack ||
                (vs_top * vc[t][e] >= kWide &&
                 (!MASK || top[t][e] > __uint_as_float(0xFF800000u)));
      }
    if (__any_sync(0xffffffffu, over)) {
      // the rows' maxima and factors move (of all rows: each alone moves more often): what
      // was summed is rescaled
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = top[t][e];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          float vs = vs_top;
          if (MASK) {  // of the blocks that the row sees keys of
            vs = 0.0f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int k = key0 + 16 * u, h = hi[t][e];
              if (k < h && (window == 0 || k + 15 >= h - window)) vs = fmaxf(vs, vscale[u]);
            }
          }
          const float by = fminf(m[t][e] - x, 0.0f);
          const float to = factor_for(vc[t][e], vs);
          f[e] = exp2_fast(by + static_cast<float>(shift_of(vc[t][e]) - shift_of(to)));
          l[t][e] *= exp2_fast(by);
          m[t][e] = by < 0.0f ? x : m[t][e];
          vc[t][e] = to;
        }
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          o[t][j][0] *= f[0];
          o[t][j][1] *= f[1];
          o[t][j][2] *= f[0];
          o[t][j][3] *= f[1];
        }
      }
    }
    // probabilities; those of the values carry the block's scale (NaN scales stay NaN,
    // but only where a key is seen)
    uint32_t pb[2][NT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float vf0 = vscale[u] * vc[t][0], vf1 = vscale[u] * vc[t][1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p0 = exp2_fast(s[u][t][2 * h] - m[t][0]);
          const float p1 = exp2_fast(s[u][t][2 * h + 1] - m[t][1]);
          l[t][0] += p0;
          l[t][1] += p1;
          float y0 = p0 * vf0, y1 = p1 * vf1;
          if (MASK) {
            y0 = p0 == 0.0f ? 0.0f : y0;
            y1 = p1 == 0.0f ? 0.0f : y1;
          }
          const __half2 ph = __floats2half2_rn(y0, y1);
          pb[u][t][h] = transpose8x8(*reinterpret_cast<const uint32_t*>(&ph));
        }
      }
    }
    // keys past the end of the sequence: their codes are whatever lies there, times 0
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t vr[4][D / 32];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint32_t a = at + v_at[h & 1] + u * (16 * D) + (h >> 1) * (8 * D);
        if constexpr (D == 128) {
          const uint4 x = lds128(a);
          vr[h][0] = x.x;
          vr[h][1] = x.y;
          vr[h][2] = x.z;
          vr[h][3] = x.w;
        } else {
          const uint2 x = lds64(a);
          vr[h][0] = x.x;
          vr[h][1] = x.y;
        }
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        // four dimensions of tokens k = 2c, 2c + 1 and 2c + 8, 2c + 9
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half == 0 ? 0x5410u : 0x7632u;  // d0 d1 | d2 d3 of both tokens
          uint32_t a0, a1, a2, a3;
          halves_of(__byte_perm(vr[0][w], vr[1][w], sel), low, a0, a1);
          halves_of(__byte_perm(vr[2][w], vr[3][w], sel), low, a2, a3);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma_f16(o[t][2 * w + half], a0, a1, a2, a3, pb[u][t][0], pb[u][t][1]);
        }
      }
    }
  };
  int step = warp;
#pragma unroll 1
  for (; step < steps; step += kWarps) {
    if (!(ok = wait_warp_short(&full[warp][stage], phase, p.wait_ns, p.status, 91))) break;
    if (32 * step < all_lo || 32 * step + 32 > all_hi)
      process(step, std::true_type());
    else
      process(step, std::false_type());
    __syncwarp();  // every lane has read the stage
    if (lane == 0 && step + STAGES * kWarps < steps)
      fetch(step + STAGES * kWarps, stage, [&](int i) { return s_page[i]; });
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1u;
    }
  }

  if (!ok) {
    // The copies under way end before the rings are written over, and the rows are NaN.
    const uint64_t t0 = global_timer_ns();
    for (int i = 0; i < STAGES && step + i * kWarps < steps; ++i) {
      const int s = stage + i;
      drain_bar(&full[warp][s % STAGES], s < STAGES ? phase : phase ^ 1u, t0);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) l[t][0] = l[t][1] = __uint_as_float(0x7FC00000u);
  }

  // --------------------------------------------------------------- join the warps
  // Every warp leaves its sums as they lie in its lanes; behind one barrier a thread
  // takes 8 neighbouring dimensions of a row (a lane's, half an eighth or a whole
  // one) and adds the warps' with their factors.
  __syncthreads();  // all rings are read
  float* const mine_o = s_o + warp * (NT * KS * 4 * 32) + lane;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        mine_o[((t * 2 + (e & 1)) * (D / 8) + 2 * j + (e >> 1)) * 32] = o[t][j][e];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 4);
      l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 8);
      l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 16);
      if (r == 0) {
        s_m[warp][8 * t + 2 * c + e] = m[t][e];
        s_l[warp][8 * t + 2 * c + e] = l[t][e];
        s_d[warp][8 * t + 2 * c + e] = static_cast<float>(shift_of(vc[t][e]));
      }
    }
  }
  __syncthreads();
  constexpr int PARTS = D / 64;  // threads for a lane's dimensions of one row
  for (int i = threadIdx.x; i < NT * 64 * PARTS; i += 32 * kWarps) {
    const int src = i & 31, te = (i >> 5) % (2 * NT), piece = i / (64 * NT);
    const int at = 8 * (te >> 1) + 2 * (src & 3) + (te & 1);  // row of the group
    const int row = row0 + at;
    if (row >= rows) continue;
    float top = kLow, sum = 0.0f, most = -119.0f, f[kWarps], x[8] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][at]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float by = s_m[w][at] - top;
      sum += s_l[w][at] * exp2_fast(by);
      f[w] = by + s_d[w][at];  // log2 of a warp's sums against 2^7
      most = fmaxf(most, f[w]);
    }
    most = ceilf(most);
    const float undo = undo_factor(static_cast<int>(most));
#pragma unroll
    for (int w = 0; w < kWarps; ++w) f[w] = exp2_fast(f[w] - most);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int d = 0; d < 8; ++d)
        x[d] = fmaf(s_o[w * (NT * KS * 4 * 32) + (te * (D / 8) + 8 * piece + d) * 32 + src], f[w],
                    x[d]);
    const int sr = src >> 2;
    const int dim = (D == 128 ? ((sr & 1) * 4 + (sr >> 1)) * 16 : sr * 8) + 8 * piece;
    const unsigned tok = static_cast<unsigned>(row) / p.group;
    const int64_t t = q0 + tok;
    const int head = kvh * p.group + static_cast<int>(row - tok * p.group);
    const int64_t slot = (static_cast<int64_t>(part) * p.tokens + t) * p.heads + head;
    // the average before its size: no value on the way is larger than the values are
    const float norm = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int d = 0; d < 8; ++d) x[d] = x[d] * norm * undo;
    if (single) {
      uint4 v;
      T* w = reinterpret_cast<T*>(&v);
#pragma unroll
      for (int d = 0; d < 8; ++d) w[d] = from_float<T>(x[d]);
      *reinterpret_cast<uint4*>(out + t * p.ldo + head * D + dim) = v;
    } else {
      float4* to = reinterpret_cast<float4*>(p.part_o + slot * D + dim);
      to[0] = make_float4(x[0], x[1], x[2], x[3]);
      to[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
    if (sr == 0 && piece == 0) {
      if (!single)
        p.part_ml[slot] = make_float2(top, sum);
      else if (p.lse != nullptr)
        p.lse[t * p.heads + head] =
            sum == 0.0f ? __uint_as_float(0xFF800000u) : (top + log2f(sum)) * kLn2;
    }
  }
}

// Joins the chunks of one (token, head): the largest maximum and the whole sum first,
// then every warp adds its chunks' averages by their shares of that sum, the loads of
// several under way at once.
constexpr int kJoinWarps = 8;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) kv8_join_kernel(Kv8Attn p) {
  constexpr int V = D / 32;  // values a lane
  __shared__ float s_top[kJoinWarps], s_sum[kJoinWarps];
  __shared__ float s_o[kJoinWarps][D];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x / static_cast<unsigned>(p.heads);
  const int head = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.heads));
  const int b = find_sequence(p.cu, p.batch, t, lane);
  if (b < 0) return;
  const int64_t q0 = __ldg(p.cu + b), q1 = __ldg(p.cu + b + 1), len = __ldg(p.lens + b);
  const int64_t n = q1 - q0;
  if (bad_lengths(p, q0, q1, len)) return;  // its rows are NaN already
  const int span = static_cast<int>(len) -
                   first_block_key(static_cast<int>(len), static_cast<int>(n), p.window, p.block);
  const int nc = (span + p.chunk - 1) / p.chunk;
  if (nc <= 1) return;  // written by its only chunk
  const int64_t stride = p.tokens * p.heads;
  const float2* ml = p.part_ml + t * p.heads + head;
  const float* po = p.part_o + (t * p.heads + head) * D + V * lane;
  float top = kLow, total = 0.0f;
  for (int i = threadIdx.x; i < nc; i += 32 * kJoinWarps) {
    const float2 x = ml[i * stride];
    const float most = fmaxf(top, x.x);
    total = total * exp2_fast(top - most) + x.y * exp2_fast(x.x - most);
    top = most;
  }
  const float most = warp_max(top);
  total = warp_sum(total * exp2_fast(top - most));
  if (lane == 0) {
    s_top[warp] = most;
    s_sum[warp] = total;
  }
  __syncthreads();
  top = kLow;
  total = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_top[w]);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) total += s_sum[w] * exp2_fast(s_top[w] - top);
  const float norm = total == 0.0f ? 0.0f : 1.0f / total;
  float o[V] = {};
#pragma unroll 4
  for (int i = warp; i < nc; i += kJoinWarps) {
    const float2 x = ml[i * stride];
    const float f = x.y * exp2_fast(x.x - top) * norm;
    const float* at = po + i * stride * D;
    if constexpr (V == 4) {
      const float4 v = *reinterpret_cast<const float4*>(at);
      o[0] = fmaf(v.x, f, o[0]);
      o[1] = fmaf(v.y, f, o[1]);
      o[2] = fmaf(v.z, f, o[2]);
      o[3] = fmaf(v.w, f, o[3]);
    } else {
      const float2 v = *reinterpret_cast<const float2*>(at);
      o[0] = fmaf(v.x, f, o[0]);
      o[1] = fmaf(v.y, f, o[1]);
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) s_o[warp][V * lane + j] = o[j];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += 32 * kJoinWarps) {
    float x = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) x += s_o[w][d];
    static_cast<T*>(p.out)[t * p.ldo + head * D + d] = from_float<T>(x);
  }
  if (threadIdx.x == 0 && p.lse != nullptr)
    p.lse[t * p.heads + head] =
        total == 0.0f ? __uint_as_float(0xFF800000u) : (top + log2f(total)) * kLn2;
}

// Keys a chunk: one wave of CTAs where the sequences and heads
// alone do not fill it, but no chunk so short that starting and joining it costs
// more than it spreads; where they do, chunks that even out ragged lengths.
constexpr int64_t kMinChunk = 256, kManyCtasChunk = 2048, kMaxChunk = 4096;
constexpr int64_t kMinPromptChunk = 512;
// Rows a kv head above which the tensor-memory kernel runs.  Groups of 16 rows here each
// read the codes again, mostly from L2; there the time hardly depends on the rows.
// Here and there in us, 8 sequences of 4096 keys and 8 kv heads: dim 128, 16 rows 28.9
// and 61.1, 32 rows 50.9 and 63.2, 48 rows 73.4 and 67.1; dim 64, 32 rows 27.9 and 52.6,
// 48 rows 43.7 and 55.9.  48 such sequences: dim 128, 32 rows 267 and 287, 48 rows 385 and
// 291; dim 64, 48 rows 197 and 249.
constexpr int64_t many_rows(int dim) { return dim == 64 ? 48 : 32; }

struct AttnPlan {
  bool prompt;       // kv8_prompt.cu
  int nt;            // groups of eight rows a CTA
  int64_t row_groups, chunk;
  int window;        // 0: none
  int chunks;
};

AttnPlan plan_attention(int64_t tokens, int heads, int kv_heads, int head_dim, int64_t batch,
                        int64_t max_new, int64_t max_len, int64_t window) {
  AttnPlan a;
  a.window = window < max_len ? static_cast<int>(window) : 0;  // a wider one hides nothing
  const int64_t rows = std::min(std::max<int64_t>(max_new, 1), std::max<int64_t>(tokens, 1)) *
                       (heads / kv_heads);
  a.prompt = rows > many_rows(head_dim);
  a.nt = rows <= 8 ? 1 : 2;
  a.row_groups = ceil_div(rows, 8 * a.nt);
  int64_t span = max_len;  // most keys in sight of a sequence, from a block's (at most 128) start
  if (a.window > 0) span = std::min(span, window + max_new + 128);
  span = std::max<int64_t>(span, 1);
  if (a.prompt) {
    // whole multiprocessors: split the keys only where the rows leave some idle
    const int64_t ctas = std::min(tokens * (heads / kv_heads) / kPromptRows + batch,
                                  ceil_div(rows, kPromptRows) * batch) *
                         kv_heads;
    const int64_t want = std::max<int64_t>(1, 148 / ctas);
    a.chunk = std::max(ceil_div(ceil_div(span, want), 128) * 128, kMinPromptChunk);
    a.chunks = static_cast<int>(ceil_div(span, a.chunk));
    return a;
  }
  const int64_t ctas = a.row_groups * kv_heads * batch;
  const int64_t want = 148 * ctas_sm(head_dim, a.nt) / ctas;
  a.chunk = want > 1 ? ceil_div(ceil_div(span, want), 128) * 128 : kManyCtasChunk;
  a.chunk = std::min(std::max(a.chunk, kMinChunk), kMaxChunk);
  a.chunks = static_cast<int>(ceil_div(span, a.chunk));
  return a;
}

bool attn_sizes_ok(int64_t tokens, int heads, int kv_heads, int head_dim, int64_t batch,
                   int64_t max_new, int64_t max_len, int window) {
  return tokens >= 0 && tokens <= (int64_t)1 << 24 && kv_heads >= 1 && kv_heads <= 1024 &&
         heads >= kv_heads && heads % kv_heads == 0 && heads / kv_heads <= 256 &&
         tokens * heads <= INT32_MAX - 256 &&
         (head_dim == 64 || head_dim == 128) && batch >= 1 && batch <= 65535 && max_new >= 0 &&
         max_new <= INT32_MAX && max_len >= 0 && max_len <= (int64_t)1 << 26 && window >= 0;
}

struct AttnWs {
  size_t ml_at, bytes;
};
AttnWs attn_ws(const AttnPlan& a, int64_t tokens, int heads, int head_dim) {
  AttnWs w;
  const size_t slots = a.chunks > 1 ? static_cast<size_t>(a.chunks) * tokens * heads : 0;
  w.ml_at = (slots * head_dim * 4 + 255) / 256 * 256;
  w.bytes = std::max<size_t>(256, w.ml_at + (slots * 8 + 255) / 256 * 256);
  return w;
}

// The codes as [pages kv_heads][block][D], in boxes of 32 tokens (16 where a page has
// no more), swizzled over a token's bytes.
template <int D>
bool page_map(CUtensorMap* map, const int8_t* codes, const Kv8Attn& p) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(p.block),
                              static_cast<cuuint64_t>(p.pages) * p.kv_heads};
  const cuuint64_t strides[2] = {D, static_cast<cuuint64_t>(D) * p.block};
  const cuuint32_t box[3] = {D, static_cast<cuuint32_t>(std::min(p.block, 32)), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t*>(codes), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
int launch_join(const Kv8Attn& p, cudaStream_t stream) {
  note_launch();
  return launch_pdl(kv8_join_kernel<T, D>, dim3(static_cast<unsigned>(p.tokens * p.heads)),
                    dim3(32 * kJoinWarps), 0, stream, p) == cudaSuccess
             ? PIQ_OK
             : PIQ_ERR_CUDA;
}

template <typename T, int D>
int launch_attention(const Kv8Attn& p, const AttnPlan& a, cudaStream_t stream) {
  if (a.prompt) {
    const int rc = launch_prompt<T, D>(p, stream);
    if (rc != PIQ_OK) return rc;
    return a.chunks == 1 ? PIQ_OK : launch_join<T, D>(p, stream);
  }
  void (*kern)(CUtensorMap, CUtensorMap, Kv8Attn) =
      a.nt == 1 ? kv8_chunk_kernel<T, D, 1> : kv8_chunk_kernel<T, D, 2>;
  const unsigned gx = static_cast<unsigned>(a.row_groups * p.kv_heads);
  constexpr int smem = kWarps * ring_bytes(D) + 1024;
  CUtensorMap mk, mv;
  if (!page_map<D>(&mk, p.kc, p) || !page_map<D>(&mv, p.vc, p)) return PIQ_ERR_INVALID_ARG;
  static std::atomic<bool> set[2][64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PIQ_ERR_CUDA;
  std::atomic<bool>* done = dev < 64 ? &set[a.nt - 1][dev] : nullptr;
  if (done == nullptr || !done->load(std::memory_order_acquire)) {
    const int rc =
        cuda_rc(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    if (rc != PIQ_OK) return rc;
    if (done != nullptr) done->store(true, std::memory_order_release);
  }
  note_launch();
  if (launch_pdl(kern, dim3(gx, a.chunks, p.batch), dim3(32 * kWarps), smem, stream, mk, mv, p) !=
      cudaSuccess)
    return PIQ_ERR_CUDA;
  return a.chunks == 1 ? PIQ_OK : launch_join<T, D>(p, stream);
}

}  // namespace

bool kv8_cache_ok(const void* kc, const void* vc, const void* ks, const void* vs, int64_t pages,
                  int heads, int head_dim, int block);
bool kv8_table_ok(const void* cu, const void* lens, int64_t batch, const void* table,
                  int64_t width, int64_t ldt, const void* status);

}  // namespace piq

extern "C" {
using namespace piq;

int piq_kv8_attention_workspace_bytes(int64_t tokens, int heads, int kv_heads, int head_dim,
                                      int64_t batch, int64_t max_new, int64_t max_len,
                                      int window, size_t* bytes) {
  if (bytes == nullptr ||
      !attn_sizes_ok(tokens, heads, kv_heads, head_dim, batch, max_new, max_len, window))
    return PIQ_ERR_INVALID_ARG;
  const AttnPlan a =
      plan_attention(tokens, heads, kv_heads, head_dim, batch, max_new, max_len, window);
  *bytes = attn_ws(a, tokens, heads, head_dim).bytes;
  return PIQ_OK;
}

int piq_kv8_attention(const void* q, int dtype, int64_t tokens, int64_t ldq, int heads,
                      const int32_t* cu_q, const int32_t* lens, int64_t batch,
                      const int32_t* block_table, int64_t table_width, int64_t ldt,
                      const int8_t* k_codes, const int8_t* v_codes, const float* k_scale,
                      const float* v_scale, int64_t pages, int kv_heads, int head_dim, int block,
                      float scale, int window, int64_t max_new, int64_t max_len, void* out,
                      int64_t ldo, float* lse, int32_t* status, void* workspace,
                      size_t ws_bytes, void* stream) {
  if ((dtype != PIQ_BF16 && dtype != PIQ_FP16) ||
      !attn_sizes_ok(tokens, heads, kv_heads, head_dim, batch, max_new, max_len, window) ||
      !kv8_cache_ok(k_codes, v_codes, k_scale, v_scale, pages, kv_heads, head_dim, block) ||
      !kv8_table_ok(cu_q, lens, batch, block_table, table_width, ldt, status) ||
      !(std::fabs(scale) <= 0x1p127f))  // scale log2(e) is finite
    return PIQ_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(heads) * head_dim;
  if (ldq < row || ldo < row || ldq % 8 != 0 || ldo % 8 != 0) return PIQ_ERR_INVALID_ARG;
  if (tokens == 0) return PIQ_OK;
  if (q == nullptr || out == nullptr || !ptr_aligned(q, 16) || !ptr_aligned(out, 16) ||
      !ptr_aligned(lse, 4) || workspace == nullptr || !ptr_aligned(workspace, 256))
    return PIQ_ERR_INVALID_ARG;
  const AttnPlan a =
      plan_attention(tokens, heads, kv_heads, head_dim, batch, max_new, max_len, window);
  const AttnWs w = attn_ws(a, tokens, heads, head_dim);
  if (ws_bytes < w.bytes) return PIQ_ERR_WORKSPACE_TOO_SMALL;
  int rc = injected_fault();
  DeviceInfo info;
  if (rc == PIQ_OK) rc = device_info(&info);
  if (rc != PIQ_OK) return rc;
  Kv8Attn p;
  p.q = q;
  p.tokens = tokens;
  p.ldq = ldq;
  p.cu = cu_q;
  p.lens = lens;
  p.table = block_table;
  p.width = table_width;
  p.ldt = ldt;
  p.kc = k_codes;
  p.vc = v_codes;
  p.ks = k_scale;
  p.vs = v_scale;
  p.pages = pages;
  p.batch = static_cast<int>(batch);
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.block = block;
  p.group = heads / kv_heads;
  p.scale2 = scale * 1.4426950408889634f;
  p.window = a.window;
  p.max_new = max_new;
  p.max_len = max_len;
  p.chunk = static_cast<int>(a.chunk);
  p.chunks = a.chunks;
  p.out = out;
  p.ldo = ldo;
  p.lse = lse;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + w.ml_at);
  p.status = status;
  p.wait_ns = serving_wait_ns();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == PIQ_BF16)
    return head_dim == 128 ? launch_attention<__nv_bfloat16, 128>(p, a, s)
                           : launch_attention<__nv_bfloat16, 64>(p, a, s);
  return head_dim == 128 ? launch_attention<__half, 128>(p, a, s)
                         : launch_attention<__half, 64>(p, a, s);
}

}  // extern "C"
