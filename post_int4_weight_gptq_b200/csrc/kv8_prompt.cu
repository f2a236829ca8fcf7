// Attention of many new tokens over the 8-bit paged cache on the tensor cores
// (tcgen05 kind::f16, fp32 in TMEM).
//
// A CTA holds 256 query rows of one kv head, two tiles of 128 rows; rows are
// (token, head) pairs, the heads of the group fastest, so that all heads of the
// group share the keys.  Keys pass in tiles of 128:
//
//   S = Q K^T    (both fp16 in shared memory; a code is exact in fp16)
//   P = 2^(x - m) v_scale c,  x = S scale k_scale             (TMEM over S, fp16)
//   O += P V     (P from TMEM, V's codes fp16 in shared memory)
//
// with the running maximum m moved, and O rescaled, only when a score passes it
// by 2^7.  c is 2^7 over the largest value scale that the row has seen (a power of
// two, moved like m); the sum of 2^(x - m) is fp32.  The codes are widened to fp16
// as they come from the pages (no second copy of the cache exists): bytes go through
// registers to the swizzled tiles both products read.
//
// 16 warps: 0 - 3 and 4 - 7 the softmax of tile 0 and 1 (a row a thread),
// 8 - 11 widen keys and values, 12 issues the MMAs (13 - 15 only give their
// registers away).  The two tiles alternate: one tile's softmax runs while the tensor
// cores work for the other.  Every wait is bounded.
#include <algorithm>
#include <atomic>

#include "kv8_attn.cuh"

namespace piq {

namespace {

constexpr int KT = 128;      // keys a tile
constexpr int kThreads = 16 * 32;
constexpr int kGran = KT / 16;  // 16-key granules: never across a page

// fp16 A and B, fp32 D; B optionally MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// D += A B^T with A in tensor memory.
__device__ __forceinline__ void umma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// A warpgroup's registers a thread.  The block is launched with 16 warps of 128
// registers; the shares below (2 x 144 softmax, 152 widening, 72 the rest) are all
// of that.
constexpr int kRegSoftmax = 144, kRegWiden = 152, kRegIssue = 72;
static_assert(2 * kRegSoftmax + kRegWiden + kRegIssue <= 4 * 128, "more than the launch has");
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Four codes to four halves, in order.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  w ^= 0x80808080u;
  const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), off);
  const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), off);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Two floats in one register pair.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Which of a tile's keys 32 c .. 32 c + 31 lie in [from, upto).
__device__ __forceinline__ uint32_t seen(int from, int upto, int c) {
  const int a = min(max(from - 32 * c, 0), 32), b = min(max(upto - 32 * c, 0), 32);
  const uint32_t below = b == 32 ? 0xFFFFFFFFu : (1u << b) - 1u;
  return a == 32 ? 0u : below & ~((1u << a) - 1u);
}

// The largest of a row's 128 scores (scaled), this thread's TMEM lane at ts, of the
// keys [from, upto).  Kept apart from the unmasked form, which all but a few tiles
// take: selects for every key cost as much as the rest.
__device__ __forceinline__ float row_max(uint32_t ts, float rs, const float* ks, int from,
                                         int upto) {
  const float ninf = __uint_as_float(0xFF800000u);
  float top = ninf;
#pragma unroll 1
  for (int c = 0; c < KT / 32; ++c) {
    float s[32];
    tmem_ld_32x32b_x32(ts + 32 * c, s);
    const uint32_t bits = seen(from, upto, c);
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = (bits >> i) & 1u ? s[i] : ninf;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      // a score times the (positive) scales is monotone in it
      float x = fmaxf(s[16 * g], s[16 * g + 1]), y = fmaxf(s[16 * g + 2], s[16 * g + 3]);
#pragma unroll
      for (int i = 4; i < 16; i += 4) {
        x = fmaxf(fmaxf(x, s[16 * g + i]), s[16 * g + i + 1]);
        y = fmaxf(fmaxf(y, s[16 * g + i + 2]), s[16 * g + i + 3]);
      }
      top = fmaxf(top, fmaxf(x, y) * (rs * ks[2 * c + g]));
    }
  }
  return top;
}

// The row's probabilities relative to m, summed into l2, and times the blocks'
// value scales and the row's factor as halves over the scores.
__device__ __forceinline__ void row_weights(uint32_t ts, float rs, float m, float vc,
                                            const float* ks, const float* vs, int from, int upto,
                                            uint64_t& l2) {
  const float ninf = __uint_as_float(0xFF800000u);
  const uint64_t nm2 = pack2(-m, -m);
#pragma unroll 1
  for (int c = 0; c < KT / 32; ++c) {
    float s[32];
    uint32_t w[16];
    tmem_ld_32x32b_x32(ts + 32 * c, s);
    const uint32_t bits = seen(from, upto, c);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float f = rs * ks[2 * c + g], vf = vs[2 * c + g] * vc;
      const uint64_t f2 = pack2(f, f), vf2 = pack2(vf, vf);
#pragma unroll
      for (int i = 16 * g; i < 16 * g + 16; i += 2) {
        float x0, x1, y0, y1;
        unpack2(fma2(pack2(s[i], s[i + 1]), f2, nm2), x0, x1);
        x0 = (bits >> i) & 1u ? x0 : ninf;
        x1 = (bits >> (i + 1)) & 1u ? x1 : ninf;
        const uint64_t e = pack2(exp2_fast(x0), exp2_fast(x1));
        l2 = add2(l2, e);
        unpack2(mul2(e, vf2), y0, y1);
        // 0 times the scale of a block that holds a NaN is not 0, nor times one that is
        // too large for the factor of a row that does not see it
        y0 = (bits >> i) & 1u ? y0 : 0.0f;
        y1 = (bits >> (i + 1)) & 1u ? y1 : 0.0f;
        const __half2 h = __floats2half2_rn(y0, y1);
        w[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    tmem_st_x16(ts + 16 * c, w);
  }
}

// Byte offset of 16-byte piece `piece` (dims 8 piece ..) of row `row` in a tile of
// 128 rows: halves of 64 dimensions, 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_at(int row, int piece) {
  return (piece >> 3) * (KT * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}

// 32 columns of this warp's lanes; the values are there after tmem_ld_done, which
// also keeps their uses behind the wait.
__device__ __forceinline__ void tmem_ld_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_ld_done(uint32_t (&r)[32]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]),
                 "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                 "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

// The unmasked forms of the two, 32 columns at a time: their largest score, and their
// probabilities relative to m as halves in w.  (All 128 columns in registers from one
// read, unrolled, came out slower: 315 us, the code no longer fits the instruction
// cache beside the other roles'.)
__device__ __forceinline__ float part_max(const uint32_t (&s)[32], float rs, const float* ks,
                                          float top) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const uint32_t* v = s + 16 * g;
    float x = fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]));
    float y = fmaxf(__uint_as_float(v[2]), __uint_as_float(v[3]));
#pragma unroll
    for (int i = 4; i < 16; i += 4) {
      x = fmaxf(fmaxf(x, __uint_as_float(v[i])), __uint_as_float(v[i + 1]));
      y = fmaxf(fmaxf(y, __uint_as_float(v[i + 2])), __uint_as_float(v[i + 3]));
    }
    top = fmaxf(top, fmaxf(x, y) * (rs * ks[g]));
  }
  return top;
}
__device__ __forceinline__ void part_weights(const uint32_t (&s)[32], uint32_t to, float rs,
                                             uint64_t nm2, float vc, const float* ks,
                                             const float* vs, uint64_t& la, uint64_t& lb) {
  uint32_t w[16];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const float f = rs * ks[g], vf = vs[g] * vc;
    const uint64_t f2 = pack2(f, f), vf2 = pack2(vf, vf);
#pragma unroll
    for (int i = 16 * g; i < 16 * g + 16; i += 2) {
      float x0, x1, y0, y1;
      unpack2(fma2(pack2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), f2, nm2), x0, x1);
      const uint64_t e = pack2(exp2_fast(x0), exp2_fast(x1));
      if (i & 2)
        la = add2(la, e);
      else
        lb = add2(lb, e);
      unpack2(mul2(e, vf2), y0, y1);
      const __half2 h = __floats2half2_rn(y0, y1);
      w[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  tmem_st_x16(to, w);
}

// The 32 query rows of a warp (row0 of `rows`, row `at` of the tile) to halves in
// shared memory.  Lanes go along a row, so that a load meets two or four rows' bytes
// whole (a row a lane took 5 us); every lane then takes its own row's factor: the
// positive factor of its scores in log2 units (the sign of scale2 goes into the
// halves).  A row that holds an infinity or NaN is zeros under a NaN factor.
template <typename T, int D>
__device__ __forceinline__ float stage_queries(const Kv8Attn& p, int64_t q0, int kvh, int row0,
                                               int rows, uint8_t* tile, int at, int lane) {
  constexpr int LPR = D / 8, RPL = 32 / LPR;  // lanes a row, rows a load
  Eight<T> v[LPR];
  const int piece = lane % LPR, sub = lane / LPR;
  int tok = static_cast<int>(static_cast<unsigned>(row0 + sub) / p.group);
  int head = row0 + sub - tok * p.group;  // stepped below: a division a row is slow
#pragma unroll
  for (int i = 0; i < LPR; ++i) {
    v[i].zero();
    if (row0 + i * RPL + sub < rows)
      v[i].load(static_cast<const T*>(p.q) + (q0 + tok) * p.ldq + (kvh * p.group + head) * D +
                8 * piece);
    for (head += RPL; head >= p.group; head -= p.group) ++tok;
  }
  float mine = 0.0f;
#pragma unroll
  for (int i = 0; i < LPR; ++i) {
    Largest<T> top;
    top.add(v[i]);
    uint32_t m = top.bits();
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    float mul;
    const float undo = row_exponent<T>(__uint_as_float(m), mul);
    const bool fine = undo == undo;
    if (p.scale2 < 0.0f) mul = -mul;
    float f[8];
    uint32_t w[4];
    v[i].floats(f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 h = __floats2half2_rn(f[2 * j] * mul, f[2 * j + 1] * mul);
      w[j] = fine ? *reinterpret_cast<const uint32_t*>(&h) : 0u;
    }
    *reinterpret_cast<uint4*>(tile + tile_at(at + i * RPL + sub, piece)) =
        make_uint4(w[0], w[1], w[2], w[3]);
    const float rs = undo * fabsf(p.scale2);
    // row i RPL + s of the warp is lane i RPL + s's, and lanes s LPR .. have its factor
    const float got = __shfl_sync(0xffffffffu, rs, (lane % RPL) * LPR);
    if (lane / RPL == i) mine = got;
  }
  return mine;
}

template <int D>
struct Layout {
  static constexpr int TILE = KT * D * 2;  // fp16 bytes of 128 rows
  static constexpr int K_AT = 2 * TILE, V_AT = 4 * TILE, BAR_AT = 6 * TILE;
  static constexpr int BYTES = BAR_AT + 1024 + 1024;
};

struct Shared {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], pv_done[2];
  uint64_t sc_full[4], q_full, o_done, drain;
  float ks[4][kGran], vs[4][kGran];  // scales of a tile: a ring of four, so that a slot is
                                     // rewritten only after both softmaxes have left it
  float vs_top[4];                   // the largest value scale of each (not NaN)
  uint32_t tmem;
};
static_assert(sizeof(Shared) <= 1024, "barrier area");

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) kv8_prompt_kernel(Kv8Attn p) {
  using L = Layout<D>;
  constexpr int PIECES = KT * D / 16 / 128;     // 16-code loads a thread and tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Shared& sh = *reinterpret_cast<Shared*>(smem + L::BAR_AT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_wait();
  // Bad lengths are found by the first CTA (whose item most often has no rows), over the
  // whole batch: with starts that cannot be, the search below may pass a sequence by.
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    auto bad = [&](int i) {
      return bad_lengths(p, __ldg(p.cu + i), __ldg(p.cu + i + 1), __ldg(p.lens + i));
    };
    bool any = false;
    for (int i = threadIdx.x; i < p.batch; i += blockDim.x) any |= bad(i);
    if (__syncthreads_or(any))
      for (int i = 0; i < p.batch; ++i)
        if (bad(i)) report_lengths<T, D>(p, i, __ldg(p.cu + i), __ldg(p.cu + i + 1));
  }
  // ------------------------------------------------------------- which rows
  // Items of 256 rows are numbered without the lengths: sequence b's start at
  // floor(cu[b] group / 256) + b.  The last ones, which see most keys, go first.
  const int kvh = blockIdx.x % p.kv_heads;
  const int64_t item = (gridDim.x - 1 - blockIdx.x) / p.kv_heads;
  const int part = blockIdx.y;
  int b;
  {
    int lo = 0, hi = p.batch;
    while (hi > lo) {
      const int step = (hi - lo + 31) / 32;
      const int probe = min(lo + step * lane + step - 1, hi - 1);
      const int64_t start = static_cast<int64_t>(__ldg(p.cu + probe)) * p.group / kPromptRows + probe;
      const unsigned votes = __ballot_sync(0xffffffffu, start <= item);
      const int run = __ffs(~votes) - 1;
      if (run < 0) {
        lo = hi;
        break;
      }
      const int nlo = min(lo + step * run, hi);
      hi = min(nlo + step - 1, hi);
      lo = nlo;
    }
    b = lo - 1;
  }
  if (b < 0) return;
  const int64_t q0 = __ldg(p.cu + b), q1 = __ldg(p.cu + b + 1), seq_len = __ldg(p.lens + b);
  if (q0 == q1) return;
  const int64_t first_row = (item - (q0 * p.group / kPromptRows + b)) * kPromptRows;
  if (bad_lengths(p, q0, q1, seq_len)) return;
  const int n = static_cast<int>(q1 - q0), len = static_cast<int>(seq_len);
  const int rows = n * p.group;
  if (first_row >= rows) return;
  const int row0 = static_cast<int>(first_row);
  const int nq = rows - row0 > 128 ? 2 : 1;  // tiles with rows in them
  // ------------------------------------------------------------- which keys
  const int origin = first_block_key(len, n, p.window, p.block);
  const int c0 = origin + part * p.chunk;
  if (c0 >= len) return;
  const int c1 = c0 + min(p.chunk, len - c0);
  const bool single = len - origin <= p.chunk;
  const int first_tok = static_cast<int>(static_cast<unsigned>(row0) / p.group);
  const int last_tok =
      static_cast<int>(static_cast<unsigned>(min(row0 + kPromptRows, rows) - 1) / p.group);
  const int see_lo = p.window > 0 ? max(len - n + first_tok + 1 - p.window, 0) : 0;
  const int k0 = max(c0, see_lo & ~15);
  const int k1 = min(c1, len - n + last_tok + 1);
  const int nt = k1 > k0 ? (k1 - k0 + KT - 1) / KT : 0;
  const int shift = __ffs(p.block) - 1;
  const int32_t* table = p.table + b * p.ldt;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.k_full[i], 4);
      mbar_init(&sh.v_full[i], 4);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sh.sc_full[i], 1);
    mbar_init(&sh.q_full, 4 * nq);
    mbar_init(&sh.o_done, 1);
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // behind the allocation: a kernel that starts early must not hold tensor memory that
  // this one still waits for
  pdl_launch_dependents();

  if (warp >= 12) {
    // --------------------------------------------------------------- MMA issuer
    fewer_registers<kRegIssue>();
    if (warp == 12 && lane == 0 && nt > 0) {
      constexpr uint32_t id_s = idesc_f16(128, KT, false), id_o = idesc_f16(128, D, true);
      const uint32_t qa = smem_u32(smem);
      auto scores = [&](int t, int st) {
        const uint32_t a = qa + t * L::TILE, k = qa + L::K_AT + st * L::TILE;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * (KT * 128) + (kk & 3) * 32;
          umma_bf16(tmem + t * KT, smem_desc(a + off, 16, 1024, kLayoutSw128),
                   smem_desc(k + off, 16, 1024, kLayoutSw128), id_s, kk != 0);
        }
        umma_commit(&sh.s_full[t]);
      };
      bool ok = wait_bar(&sh.q_full, 0, p.wait_ns, p.status, 70) &&
                wait_bar(&sh.k_full[0], 0, p.wait_ns, p.status, 71);
      const bool began = ok;
      if (ok) {
        tc_fence_after();
        for (int t = 0; t < nq; ++t) scores(t, 0);
        umma_commit(&sh.k_empty[0]);
      }
      for (int j = 0; j < nt && ok; ++j) {
        const int st = j & 1;
        if (!(ok = wait_bar(&sh.v_full[st], (j >> 1) & 1, p.wait_ns, p.status, 72))) break;
        const bool more = j + 1 < nt;
        if (more &&
            !(ok = wait_bar(&sh.k_full[st ^ 1], ((j + 1) >> 1) & 1, p.wait_ns, p.status, 73)))
          break;
        for (int t = 0; t < nq; ++t) {
          if (!(ok = wait_bar(&sh.p_full[t], j & 1, p.wait_ns, p.status, 74))) break;
          tc_fence_after();
          const uint32_t v = qa + L::V_AT + st * L::TILE;
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk)
            umma_f16_ts(tmem + 2 * KT + t * D, tmem + t * KT + kk * 8,
                        smem_desc(v + kk * 2048, KT * 128, 1024, kLayoutSw128), id_o,
                        (j | kk) != 0);
          umma_commit(&sh.pv_done[t]);
          if (more) {
            // The next scores go over the P that this product reads: MMAs on other
            // accumulators are not ordered behind it, so its end is waited for.
            if (!(ok = wait_bar(&sh.pv_done[t], j & 1, p.wait_ns, p.status, 76))) break;
            scores(t, st ^ 1);
          }
        }
        if (!ok) break;
        umma_commit(&sh.v_empty[st]);
        if (more) umma_commit(&sh.k_empty[st ^ 1]);
      }
      // the end of everything; the arrival is in before the barrier's memory goes.  After a
      // wait that gave up, the same on a barrier that tells nobody that O is there.
      if (began) {
        uint64_t* const end = ok ? &sh.o_done : &sh.drain;
        umma_commit(end);
        drain_bar(end, 0, global_timer_ns());
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------ widening keys and values
    more_registers<kRegWiden>();
    // A granule of 16 keys is one run of 16 D bytes; the 128 threads take 128 / D
    // of them at a time, 16 bytes each.  Four lanes share a key's 64 dimensions and
    // the next four the key after it, whose swizzle puts their halves into the other
    // banks.
    constexpr int GPL = 128 / D;                       // granules a load
    const int tid = threadIdx.x - 256;
    const int piece = tid & 3, key = ((tid >> 2) & 1) + 2 * ((tid >> 3) & 7);
    const int gsel = D == 128 ? 0 : tid >> 6, half = D == 128 ? tid >> 6 : 0;
    const int from = key * D + half * 64 + piece * 16;  // in the granule
    const uint32_t to0 = tile_at(gsel * 16 + key, half * 8 + 2 * piece),
                   to1 = tile_at(gsel * 16 + key, half * 8 + 2 * piece + 1);
    uint4 kr[PIECES], vr[PIECES];
    // Granule `lane & 7` of a tile: its table entry is fetched two tiles ahead, its
    // scales one, so that neither is waited for.
    int entry = 0;
    int64_t base = 0;
    float gks = 0.0f, gvs = 0.0f;
    auto fetch = [&](int j) {
      const int k = k0 + j * KT + 16 * (lane & 7);
      entry = k < k1 ? __ldg(table + (k >> shift)) : -2;  // -2: no such keys
    };
    auto look = [&](int j) {
      int page = 0;
      gks = gvs = entry == -2 ? 0.0f : __uint_as_float(0x7FC00000u);
      if (entry >= 0 && entry < p.pages) {
        page = entry;
        gks = __ldg(p.ks + static_cast<int64_t>(page) * p.kv_heads + kvh);
        gvs = __ldg(p.vs + static_cast<int64_t>(page) * p.kv_heads + kvh);
      } else if (entry != -2) {
        note_status(p.status, PIQ_ERR_INVALID_ARG, b);
      }
      const int off = (k0 + j * KT + 16 * (lane & 7)) & (p.block - 1);
      base = ((static_cast<int64_t>(page) * p.kv_heads + kvh) * p.block + off) * D;
    };
    auto load = [&](const int8_t* codes, uint4 (&reg)[PIECES]) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        reg[i] = __ldg(reinterpret_cast<const uint4*>(
            codes + __shfl_sync(0xffffffffu, base, i * GPL + gsel) + from));
    };
    auto store = [&](uint8_t* tile, const uint4 (&reg)[PIECES]) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const uint2 x = widen4(reg[i].x), y = widen4(reg[i].y), z = widen4(reg[i].z),
                    w = widen4(reg[i].w);
        *reinterpret_cast<uint4*>(tile + to0 + i * GPL * 2048) = make_uint4(x.x, x.y, y.x, y.y);
        *reinterpret_cast<uint4*>(tile + to1 + i * GPL * 2048) = make_uint4(z.x, z.y, w.x, w.y);
      }
    };
    fetch(0);
    look(0);
    fetch(1);
    if (nt > 0) {
      load(p.kc, kr);
      load(p.vc, vr);
    }
    for (int j = 0; j < nt; ++j) {
      const int st = j & 1, slot = j & 3;
      const float tks = gks, tvs = gvs;
      look(j + 1);
      fetch(j + 2);
      if (!wait_warp(&sh.k_empty[st], ((j >> 1) & 1) ^ 1u, p.wait_ns, p.status, 83)) break;
      if (warp == 8) {
        float top = fmaxf(tvs, 0.0f);  // lanes l and l + 8 hold the same granule
#pragma unroll
        for (int o = 1; o < kGran; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane < kGran) {
          sh.ks[slot][lane] = tks;
          sh.vs[slot][lane] = tvs;
        }
        if (lane == 0) sh.vs_top[slot] = top;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.sc_full[slot]);
      }
      store(smem + L::K_AT + st * L::TILE, kr);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.k_full[st]);
      if (j + 1 < nt) load(p.kc, kr);
      if (!wait_warp(&sh.v_empty[st], ((j >> 1) & 1) ^ 1u, p.wait_ns, p.status, 84)) break;
      store(smem + L::V_AT + st * L::TILE, vr);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.v_full[st]);
      if (j + 1 < nt) load(p.vc, vr);
    }
  } else {
    // ------------------------------------------------------------------ softmax
    more_registers<kRegSoftmax>();
    if (warp < 4 * nq) {
      const unsigned row = row0 + threadIdx.x;
      const bool live = row < static_cast<unsigned>(rows);
      const unsigned rel = (live ? row : 0u) / p.group;
      const int64_t tok = q0 + rel;
      const int head = kvh * p.group + static_cast<int>((live ? row : 0u) - rel * p.group);
      const float rs = stage_queries<T, D>(p, q0, kvh, row0 + 32 * warp, rows,
                                           smem + (warp >> 2) * L::TILE, 32 * (warp & 3), lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);
      const int t = warp >> 2;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t ts = tmem + lanes + t * KT, to = tmem + lanes + 2 * KT + t * D;
      // Keys [lo, hi) are this row's, of those before the part's end: with a window the
      // tiles start where it does, and the last one may reach into the next part.
      const int end = len - n + static_cast<int>(rel) + 1;
      const int hi = live ? min(end, c1) : 0;
      const int lo = p.window > 0 ? end - p.window : 0;
      float m = kLow, vc = kFirstFactor;
      uint64_t l2 = 0;  // the sum, even and odd keys
      bool ok = true;
      for (int j = 0; j < nt; ++j) {
        const int slot = j & 3;
        const int key0 = k0 + j * KT;
        if (!(ok = wait_warp(&sh.sc_full[slot], (j >> 2) & 1, p.wait_ns, p.status, 77))) break;
        if (!(ok = wait_warp(&sh.s_full[t], j & 1, p.wait_ns, p.status, 78))) break;
        tc_fence_after();
        // keys [from, to) of the tile are seen
        const int from = max(lo - key0, 0), upto = min(max(hi - key0, 0), KT);
        const bool mask = __any_sync(0xffffffffu, from > 0 || upto < KT);
        const float *ks = sh.ks[slot], *vs = sh.vs[slot];
        // The rows' running maxima and factors move (and O is rescaled) when a score passes
        // one by 2^7 or a row sees keys of a block whose scale is too large for its factor;
        // those of the whole warp, as each row alone moves more often (298 against 289 us
        // for two chunks of 2048 tokens behind 2048, 32 heads on 8).
        auto move = [&](float top) {
          float wide = sh.vs_top[slot];
          if (!__any_sync(0xffffffffu,
                          top > m + kSlack || (wide * vc >= kWide && (!mask || upto > from))))
            return true;
          if (mask) {
            wide = 0.0f;
#pragma unroll 1
            for (int g = 0; g < kGran; ++g)
              if (16 * g < upto && 16 * g + 16 > from) wide = fmaxf(wide, vs[g]);
          }
          const float by = fminf(m - top, 0.0f), to_c = factor_for(vc, wide);
          const float f = exp2_fast(by);
          const float fo = exp2_fast(by + static_cast<float>(shift_of(vc) - shift_of(to_c)));
          m = by < 0.0f ? top : m;
          vc = to_c;
          l2 = mul2(l2, pack2(f, f));
          if (j == 0 || !__any_sync(0xffffffffu, fo != 1.0f)) return true;
          if (!wait_warp(&sh.pv_done[t], (j - 1) & 1, p.wait_ns, p.status, 79)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            float o[16];
            uint32_t w[16];
            tmem_ld_32x32b_x16(to + 16 * c, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * fo);
            tmem_st_x16(to + 16 * c, w);
          }
          return true;
        };
        if (mask) {
          if (!(ok = move(row_max(ts, rs, ks, from, upto)))) break;
          row_weights(ts, rs, m, vc, ks, vs, from, upto, l2);
        } else {
          // two buffers of 32 columns: one is on its way while the other is worked on
          uint32_t sa[32], sb[32];
          float top = __uint_as_float(0xFF800000u);
          tmem_ld_start(ts, sa);
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            tmem_ld_wait();
            tmem_ld_done(sa);
            tmem_ld_start(ts + 32 * (c + 1), sb);
            top = part_max(sa, rs, ks + 2 * c, top);
            tmem_ld_wait();
            tmem_ld_done(sb);
            tmem_ld_start(ts + 32 * ((c + 2) & 3), sa);  // at last the first ones again
            top = part_max(sb, rs, ks + 2 * c + 2, top);
          }
          tmem_ld_wait();
          tmem_ld_done(sa);
          if (!(ok = move(top))) break;
          const uint64_t nm2 = pack2(-m, -m);
          uint64_t lb = 0;
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            tmem_ld_start(ts + 32 * (c + 1), sb);
            part_weights(sa, ts + 16 * c, rs, nm2, vc, ks + 2 * c, vs + 2 * c, l2, lb);
            tmem_ld_wait();
            tmem_ld_done(sb);
            if (c == 0) tmem_ld_start(ts + 64, sa);
            part_weights(sb, ts + 16 * c + 16, rs, nm2, vc, ks + 2 * c + 2, vs + 2 * c + 2, l2, lb);
            tmem_ld_wait();
            tmem_ld_done(sa);
          }
          l2 = add2(l2, lb);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[t]);
      }
      // ------------------------------------------------------------------- result
      if (ok && nt > 0) ok = wait_warp(&sh.o_done, 0, p.wait_ns, p.status, 80);
      tc_fence_after();
      float la, lb;
      unpack2(l2, la, lb);
      const float l = ok ? la + lb : __uint_as_float(0x7FC00000u);
      const float norm = l == 0.0f ? 0.0f : 1.0f / l;
      const float undo = undo_factor(shift_of(vc));
      const int64_t slot = (static_cast<int64_t>(part) * p.tokens + tok) * p.heads + head;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        float o[16];
        __syncwarp();
        if (ok && nt > 0) {
          tmem_ld_32x32b_x16(to + 16 * c, o);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0.0f;
        }
        // the average before its size: no value on the way is larger than the values are
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = o[i] * norm * undo;
        if (live && single) {
          T* at = static_cast<T*>(p.out) + tok * p.ldo + head * D + 16 * c;
          uint4 v[2];
          T* w = reinterpret_cast<T*>(v);
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = from_float<T>(o[i]);
          reinterpret_cast<uint4*>(at)[0] = v[0];
          reinterpret_cast<uint4*>(at)[1] = v[1];
        } else if (live) {
          float4* at = reinterpret_cast<float4*>(p.part_o + slot * D + 16 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            at[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      if (live) {
        if (!single)
          p.part_ml[slot] = make_float2(m, l);
        else if (p.lse != nullptr)
          p.lse[tok * p.heads + head] =
              l == 0.0f ? __uint_as_float(0xFF800000u) : (m + log2f(l)) * kLn2;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

template <typename T, int D>
int launch_prompt(const Kv8Attn& p, cudaStream_t stream) {
  static std::atomic<bool> set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PIQ_ERR_CUDA;
  if (dev >= 64 || !set[dev].load(std::memory_order_acquire)) {
    const int rc = cuda_rc(cudaFuncSetAttribute(
        kv8_prompt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::BYTES));
    if (rc != PIQ_OK) return rc;
    if (dev < 64) set[dev].store(true, std::memory_order_release);
  }
  const int64_t items = p.tokens * p.group / kPromptRows + p.batch;
  note_launch();
  return launch_pdl(kv8_prompt_kernel<T, D>,
                    dim3(static_cast<unsigned>(items * p.kv_heads), p.chunks), dim3(kThreads),
                    static_cast<size_t>(Layout<D>::BYTES), stream, p) == cudaSuccess
             ? PIQ_OK
             : PIQ_ERR_CUDA;
}

template int launch_prompt<__nv_bfloat16, 64>(const Kv8Attn&, cudaStream_t);
template int launch_prompt<__nv_bfloat16, 128>(const Kv8Attn&, cudaStream_t);
template int launch_prompt<__half, 64>(const Kv8Attn&, cudaStream_t);
template int launch_prompt<__half, 128>(const Kv8Attn&, cudaStream_t);

}  // namespace piq
