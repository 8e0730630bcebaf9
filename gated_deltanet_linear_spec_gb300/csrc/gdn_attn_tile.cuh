// gdn_attn_tile.cuh -- attention of 128-query tiles on tcgen05: what the kernels of long rows and of shared prefixes share.
//
// A tile of M = 128 queries stands in shared memory, 64 cached tokens a step:
//   S = Q K^T (128 x 64, fp32 in TMEM),  P = 2^(scale log2e (S - m)) (bf16, over S in TMEM),
//   O += P V (128 x d, fp32 in TMEM; A = P from TMEM, B = V read MN-major from its [token][d] tile);
// a thread of 128 takes a query's softmax (gdn_attn_prompt.cu says how they work together, and what was measured).
#pragma once

#include "gdn_tma.cuh"

namespace gdn {
namespace tile {

constexpr int kTN = 64;         // cached tokens of a step
constexpr float kGrow = 16.f;   // log2 of how far scores may outgrow the maximum that weights refer to

template <int D>
struct Cfg {
  static constexpr int kTiles = D <= 128 ? 2 : 1;                    // query tiles of a CTA
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kThreads = 128 * (kTiles + 1);
  static constexpr uint32_t kQ = 128 * D * 2;                        // bytes of a query tile
  static constexpr uint32_t kKv = kTN * D * 2;                       // bytes of a K or V tile
  static constexpr int kPhases = D <= 128 ? 4 : 2;                   // K and V pairs in the ring
  static constexpr int kRing = 2 * kPhases;                          // K and V tiles in turn
  static constexpr uint32_t kSmem = kTiles * kQ + kRing * kKv;
  static constexpr int kO = 256;  // first O column of TMEM; scores of tile i (buffer i) from 128 i (64 i) on
  static_assert(kSmem + 4096 <= 232448, "shared memory");
};

// Some of queries [pmin, pmax] does not see some token of [b, b + kTN).
__device__ __forceinline__ bool in_part(const AttnLaunch& p, int b, int pmin, int pmax) {
  return b + kTN - 1 > pmin || (p.window > 0 && b <= pmax - p.window && b + kTN - 1 >= p.sinks);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pack2f(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return __uint_as_float(r);
}
// acc + 0 x, a bf16 pair: stays zero, of either sign, while all x are finite, and is NaN from then on.
__device__ __forceinline__ uint32_t note2(uint32_t x, uint32_t acc) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
  return r;
}
// D (TMEM) += A (TMEM) B: A's row m is lane m, two bf16 of K per column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate));
}

// S = Q K^T of a query tile with the K tile of a ring phase, into TMEM column `to`.
template <int D>
__device__ __forceinline__ void s_products(uint32_t smem, uint32_t tile, uint32_t phase, uint32_t to) {
  using C = Cfg<D>;
  const uint64_t q = tc::sdesc(smem + tile * C::kQ, 1024);
  const uint64_t k = tc::sdesc(smem + C::kTiles * C::kQ + 2 * phase * C::kKv, D / 64 * 1024);
#pragma unroll
  for (int s = 0; s < D / 16; ++s)
    tc::mma(to, q + ((s >> 2) * 16384 + (s & 3) * 32) / 16, k + ((s >> 2) * 1024 + (s & 3) * 32) / 16,
            tc::idesc_bf16(128, kTN), s > 0);
}
// O += P V of a query tile with the V tile of a ring phase; the weights stand from TMEM column `from` on, with PAIR what
// their first 8 bits leave from column `from` + 32 on.
template <int D, bool PAIR = false>
__device__ __forceinline__ void pv_products(uint32_t smem, uint32_t tile, uint32_t phase, uint32_t from, bool onto) {
  using C = Cfg<D>;
  const uint64_t v = tc::sdesc_lbo(smem + C::kTiles * C::kQ + (2 * phase + 1) * C::kKv, 1024, D / 64 * 1024);
#pragma unroll
  for (int s = 0; s < kTN / 16; ++s) {
    const uint64_t b = v + s * 2 * (D / 64) * 1024 / 16;
    mma_ts(C::kO + tile * D, from + s * 8, b, tc::idesc_bf16_bmn(128, D), s == 0 ? (uint32_t)onto : 1u);
    if (PAIR) mma_ts(C::kO + tile * D, from + 32 + s * 8, b, tc::idesc_bf16_bmn(128, D), 1u);
  }
}

// 32 columns of this thread's TMEM lane: the load is on its way until ld_wait, which the values pass through.
__device__ __forceinline__ void ld_begin(uint32_t a, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a));
}
__device__ __forceinline__ void ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two 32-bit floats at once.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Bits [0, n) of a run of words.
__device__ __forceinline__ uint32_t low_bits(int n, int word) {
  const int k = min(max(n - 32 * word, 0), 32);
  return k == 32 ? 0xffffffffu : (1u << k) - 1u;
}

// The tokens of [b, b + 64) that a query at `pos` sees, a bit each.
__device__ __forceinline__ void visible(const AttnLaunch& p, int b, int pos, uint32_t have, bool all_pages, int bshift,
                                        uint32_t (&vis)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t x = low_bits(pos + 1 - b, i);
    if (p.window > 0) x &= ~low_bits(pos - p.window + 1 - b, i) | low_bits(p.sinks - b, i);
    if (!all_pages) {
      uint32_t pages = 0;
      for (int c = 0; c < 32; c += 16)
        if (have >> ((32 * i + c) >> bshift) & 1u) pages |= 0xffffu << c;
      x &= pages;
    }
    vis[i] = x;
  }
}

// Hides the scores of tokens that the query does not see.
__device__ __forceinline__ void hide(uint32_t (&r)[32], uint32_t vis) {
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = vis >> i & 1u ? r[i] : 0xff800000u;
}

// The weights 2^(sl2 s + ms) of 32 scores as 16 bf16 pairs; added to sum.  With PAIR they are cut to their first 8 bits, and `low`
// takes what that leaves, below 2^-7 of the weight and rounded to 8 bits: off by 2^-16 of the weight at most.  (Rounding
// the first term too would make it 2^-17, for 2 us of 164 where units have two query tiles and 1.4 of 39 where they have one.)
template <bool PAIR = false>
__device__ __forceinline__ void weights32(const uint32_t (&r)[32], uint64_t scale, uint64_t shift, uint64_t (&sum)[2],
                                          float* u, float* low = nullptr) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float a, b;
    unpair(fma2(pair(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), scale, shift), a, b);
    a = ex2(a);
    b = ex2(b);
    sum[i / 2 & 1] = add2(sum[i / 2 & 1], pair(a, b));
    if constexpr (PAIR) {
      u[i / 2] = __uint_as_float(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632));
      const uint64_t h = pair(__uint_as_float(__float_as_uint(a) & 0xffff0000u), __uint_as_float(__float_as_uint(b) & 0xffff0000u));
      float la, lb;
      unpair(fma2(h, pair(-1.f, -1.f), pair(a, b)), la, lb);
      low[i / 2] = pack2f(la, lb);
    } else {
      u[i / 2] = pack2f(a, b);
    }
  }
}

// O times f.
template <int D>
__device__ __forceinline__ void scale_o(uint32_t o_col, float f) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
    tc::tmem_ld32(o_col + c, o);
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] *= f;
    tc::tmem_st32(o_col + c, o);
  }
  tc::tmem_st_wait();
}

template <int D>
__device__ __forceinline__ void clear_o(uint32_t o_col) {
  float o[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) o[i] = 0.f;
#pragma unroll 1
  for (int c = 0; c < D; c += 32) tc::tmem_st32(o_col + c, o);
  tc::tmem_st_wait();
}

// Adds the listed tokens' share to O where the query, at `pos`, sees them: their weights from P (PAIR: both terms of them), their
// values from the cache.  O is complete up to the tile before; the warp's lanes go together, as TMEM loads and stores need
// them all.
template <int D, bool PAIR = false>
__device__ __forceinline__ void add_listed(const AttnLaunch& p, int trow, int h, const uint32_t* bad, int b, int pos,
                                           uint32_t p_col, uint32_t o_col) {
  const KvDev& kv = p.cache;
#pragma unroll 1
  for (int t = 0; t < kTN; ++t) {
    if (!(bad[t >> 5] >> (t & 31) & 1u)) continue;
    float weight = 0.f;
#pragma unroll
    for (int term = 0; term < (PAIR ? 2 : 1); ++term) {
      float x[8];
      uint32_t u = 0;
      tc::tmem_ld8(p_col + 32 * term + (t >> 1 & ~7), x);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((t >> 1 & 7) == i) u = __float_as_uint(x[i]);
      weight += __uint_as_float(t & 1 ? u & 0xffff0000u : u << 16);
    }
    const int tok = b + t;  // below the row's end, in a page that is not NULL
    const bool seen = tok <= pos && (p.window <= 0 || tok > pos - p.window || tok < p.sinks);
    const int page = kv.table[(int64_t)trow * kv.max_pages + tok / kv.page_size];
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(kv.v) + (int64_t)page * kv.page_stride +
                             ((int64_t)h * kv.page_size + tok % kv.page_size) * D;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float o[32];
      tc::tmem_ld32(o_col + c, o);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (seen) o[i] += weight * __bfloat162float(v[c + i]);
      tc::tmem_st32(o_col + c, o);
    }
    tc::tmem_st_wait();
  }
}

// A warp's 32 queries, from number row0 of the tile on; at: a lane's query's first element, -1 for zeros.  All loads
// are on their way at once.
template <int D>
__device__ __forceinline__ void load_queries(const AttnLaunch& p, uint8_t* qt, int row0, int64_t at) {
  constexpr int L = D / 8;  // lanes per row
  const int lane = threadIdx.x & 31, c = lane % L;
  const uint32_t base = tc::smem_addr(qt) + (c >> 3) * 16384;
#pragma unroll 4
  for (int i = 0; i < L; ++i) {
    const int r = i * (32 / L) + lane / L, row = row0 + r;
    const int64_t from = __shfl_sync(0xffffffffu, at, r);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(base + row * 128 + (((c & 7) ^ (row & 7)) << 4)),
                 "l"(static_cast<const __nv_bfloat16*>(p.q) + max(from, (int64_t)0) + 8 * c), "r"(from >= 0 ? 16 : 0)
                 : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace tile
}  // namespace gdn
