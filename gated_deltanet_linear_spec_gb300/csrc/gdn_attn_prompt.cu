// gdn_attn_prompt.cu -- attention of prompt rows over the paged cache on tcgen05 (bf16, d = 64, 128, 256).
//
// A tile of M = 128 queries is 128 consecutive (new token, q-head of the kv-head) pairs of a row, so
// the q-heads that share a kv-head share its keys and values in shared memory.  Per 64 cached tokens
//   S = Q K^T (128 x 64, fp32 in TMEM),  P = 2^(scale log2e (S - m)) (bf16, over S in TMEM),
//   O += P V (128 x d, fp32 in TMEM; A = P from TMEM, B = V read MN-major from its [token][d] tile).
// 4 d flops per score against about 4 issue slots of softmax: the tensor core bounds it once both run
// side by side.  So a CTA holds two query tiles (d <= 128; one at d = 256) with two score buffers each, and the
// next scores come up under the softmax of these.
//   warps 0-3 (and 4-7): softmax of tile 0 (1), a thread per query;
//   then a warp that issues all Q K^T, one that issues all P V, one that fetches pages by TMA, one that looks
//   after V tiles of which some query must not see some token (below).
// Measured on 8192 x 8192 (32 q-heads, 4 kv-heads, d = 128) on the way here: one warp for both products, which
// waits and issues in turn while the tensor core idles, 591 us; a warp for each, 533; rounds dealt back and
// forth (below), 471; the next item's queries fetched under the last output, 452 (1215 TFLOP/s).  128 tokens a
// step with one score buffer per tile and a thread holding all 128 scores took 488: a tile's products and softmax
// then follow one another, and what overlaps is the other tile's alone.  Of a step's 2000 cycles the products take
// 1650: Q K^T with N = 64 reads 6 KB of shared memory per instruction, 52 cycles instead of 32.
// P refers to a maximum that follows the running one only when that has grown by 2^16 or more, and lies 2^16 above
// it: no weight passes 1, so O overflows only where a sum of values does, and scaled by a power of two weights lose
// nothing until they are below 2^-110 of the largest, where fp32 ends.  So S is read once, and O is rescaled in TMEM
// next to never.
// P is rounded to bf16, half a step of 2^-8 relative per weight, as the product takes one 16-bit type;
// the sum of the weights is kept in fp32.  The error against 64 bits is 0.0020 to 0.0023 of the result's norm, with
// unrounded weights 0.0015 to 0.0017 (the output's own rounding).
//
// What a query does not see must not reach it whatever it holds, and 0 times NaN is NaN.  In a tile
// that some query sees only in part, values past the row's end are zeroed, and a token whose values hold an
// infinity or NaN is zeroed and listed; queries that do see it add its share to O by hand.
//
// Work items (row, 256 or 128 queries, kv-head), the longest of a row first, go to the CTAs in rounds, every
// other round in reverse order, so that who had the longest of one has the shortest of the next (1024 items of
// 1 to 128 steps: 443 steps at most, 434.5 on average; 497 without).  The items that are left for a last round
// are too few to fill the GPU: the cache of each is cut into up to 16 pieces, whose (m, l, o) meet in a second
// launch, in order.
#include <algorithm>
#include <type_traits>

#include "gdn_tma.cuh"

namespace gdn {

namespace {

constexpr int kTN = 64;         // cached tokens of a step
constexpr int kMaxPieces = 16;
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

struct PromptParams {
  AttnLaunch a;
  int max_pieces;  // of an item of the last round
  float* part;     // [kSms][kRows][D]
  float* stats;    // [kSms][kRows][2]
  uint64_t wait_ns;
};

struct Item {
  KvRow r;
  int q0;      // first (token, q-head) pair
  int h;
  int sink_tiles, first_tile, tiles;  // of its cached tokens, all pieces
  int pieces;  // > 1: this is one of several
  int j0, j1;  // its tiles
  int low;     // first position that some query sees behind the sinks
  int last;    // position of its last query
};

__device__ __forceinline__ int tile_at(const Item& w, int j) {
  return (j < w.sink_tiles ? j : w.first_tile + j - w.sink_tiles) * kTN;
}

// Items of row n: its query tiles times kv-heads.
template <int ROWS>
__device__ __forceinline__ int64_t items_of(const AttnLaunch& p, int n, uint32_t* st, KvRow& r) {
  if (n >= p.rows.num_seqs || !load_kv_row(p.rows, p.cache, n, r, st) || r.len * p.G <= p.few) return 0;
  return ((int64_t)r.len * p.G + ROWS - 1) / ROWS * p.cache.Hkv;
}

// How the items are dealt: `full` rounds of one per CTA, and a last one of the items left, cut into pieces.
struct Plan {
  int full, left, pieces;
};
__host__ __device__ inline Plan plan_of(int64_t items, int most) {
  Plan plan{(int)(items / kSms), (int)(items % kSms), 1};
  if (plan.left > 0) plan.pieces = most < kSms / plan.left ? most : kSms / plan.left;
  return plan;
}

// Finds items in increasing order of rounds; a warp holds 32 rows, one per lane.  All lanes call together.
template <int D>
struct Finder {
  static constexpr int ROWS = Cfg<D>::kRows;
  const AttnLaunch& p;
  int base = 0;
  int64_t before = 0;  // items of the rows before base
  int64_t mine = 0;    // items of row base + lane
  KvRow row;
  __device__ explicit Finder(const AttnLaunch& launch) : p(launch) { load(); }
  __device__ void load() { mine = items_of<ROWS>(p, base + (int)(threadIdx.x & 31), nullptr, row); }
  // CTA cta's item of a round; false: it has none
  __device__ bool find(const Plan& plan, int round, int cta, Item& w) {
    const int lane = threadIdx.x & 31;
    int64_t item = (int64_t)round * kSms + (round & 1 ? kSms - 1 - cta : cta);
    int piece = 0;
    w.pieces = 1;
    if (round == plan.full) {
      if (cta >= plan.left * plan.pieces) return false;
      w.pieces = plan.pieces;
      item = (int64_t)round * kSms + cta / plan.pieces;
      piece = cta % plan.pieces;
    }
    while (true) {
      int64_t inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, item >= before + inc - mine && item < before + inc);
      if (hit) {
        const int src = __ffs(hit) - 1;
        const int64_t at = item - before - __shfl_sync(0xffffffffu, inc - mine, src);
        w.r.bos = __shfl_sync(0xffffffffu, row.bos, src);
        w.r.len = __shfl_sync(0xffffffffu, row.len, src);
        w.r.kv = __shfl_sync(0xffffffffu, row.kv, src);
        w.r.trow = __shfl_sync(0xffffffffu, row.trow, src);
        const int blocks = (int)(((int64_t)w.r.len * p.G + ROWS - 1) / ROWS);
        w.h = (int)(at % p.cache.Hkv);
        w.q0 = (blocks - 1 - (int)(at / p.cache.Hkv)) * ROWS;  // the longest first
        const int pmin = w.r.kv - w.r.len + w.q0 / p.G;
        w.last = min(w.r.kv - w.r.len + (w.q0 + ROWS - 1) / p.G, w.r.kv - 1);
        w.low = p.window > 0 ? max(0, pmin - p.window + 1) : 0;
        w.sink_tiles = (min(p.sinks, w.low) + kTN - 1) / kTN;
        w.first_tile = max(w.low / kTN, w.sink_tiles);
        w.tiles = w.sink_tiles + w.last / kTN + 1 - w.first_tile;
        w.j0 = (int)((int64_t)w.tiles * piece / w.pieces);
        w.j1 = (int)((int64_t)w.tiles * (piece + 1) / w.pieces);
        return true;
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
      base += 32;
      if (base >= p.rows.num_seqs) return false;
      load();
    }
  }
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
// O += P V of a query tile with the V tile of a ring phase; the weights stand from TMEM column `from` on.
template <int D>
__device__ __forceinline__ void pv_products(uint32_t smem, uint32_t tile, uint32_t phase, uint32_t from, bool onto) {
  using C = Cfg<D>;
  const uint64_t v = tc::sdesc_lbo(smem + C::kTiles * C::kQ + (2 * phase + 1) * C::kKv, 1024, D / 64 * 1024);
#pragma unroll
  for (int s = 0; s < kTN / 16; ++s)
    mma_ts(C::kO + tile * D, from + s * 8, v + s * 2 * (D / 64) * 1024 / 16, tc::idesc_bf16_bmn(128, D),
           s == 0 ? (uint32_t)onto : 1u);
}

// Items of all rows; sum: one value per warp.  All threads call.
template <int ROWS, int THREADS>
__device__ int64_t count_items(const AttnLaunch& p, int64_t* sum) {
  int64_t mine = 0;
  for (int n = threadIdx.x; n < p.rows.num_seqs; n += THREADS) {
    KvRow r;
    mine += items_of<ROWS>(p, n, blockIdx.x == 0 ? p.status : nullptr, r);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if ((threadIdx.x & 31) == 0) sum[threadIdx.x >> 5] = mine;
  tc::fence_before();  // (orders the TMEM allocation too)
  __syncthreads();
  tc::fence_after();
  int64_t items = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) items += sum[i];
  return items;
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

// The weights 2^(sl2 s + ms) of 32 scores as 16 bf16 pairs; added to sum.
__device__ __forceinline__ void weights32(const uint32_t (&r)[32], uint64_t scale, uint64_t shift, uint64_t (&sum)[2],
                                          float* u) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float a, b;
    unpair(fma2(pair(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), scale, shift), a, b);
    a = ex2(a);
    b = ex2(b);
    sum[i / 2 & 1] = add2(sum[i / 2 & 1], pair(a, b));
    u[i / 2] = pack2f(a, b);
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

// Adds the listed tokens' share to O where the query, at `pos`, sees them: their weights from P, their values from
// the cache.  O is complete up to the tile before; the warp's lanes go together, as TMEM loads and stores need
// them all.
template <int D>
__device__ __forceinline__ void add_listed(const AttnLaunch& p, int trow, int h, const uint32_t* bad, int b, int pos,
                                           uint32_t p_col, uint32_t o_col) {
  const KvDev& kv = p.cache;
#pragma unroll 1
  for (int t = 0; t < kTN; ++t) {
    if (!(bad[t >> 5] >> (t & 31) & 1u)) continue;
    float x[8];
    uint32_t u = 0;
    tc::tmem_ld8(p_col + (t >> 1 & ~7), x);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((t >> 1 & 7) == i) u = __float_as_uint(x[i]);
    const float weight = __uint_as_float(t & 1 ? u & 0xffff0000u : u << 16);
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

template <int D>
struct Small {
  uint64_t full[Cfg<D>::kRing], empty[Cfg<D>::kRing];
  uint64_t checked[Cfg<D>::kPhases];  // of a V tile
  uint64_t q_ready[2], drain[2];
  uint64_t s_ready[2][2], p_ready[2][2], pv_done[2][2];  // [query tile][score buffer]
  int64_t sum[Cfg<D>::kThreads / 32];
  uint32_t bad[Cfg<D>::kPhases][2];  // listed tokens of a V tile
  uint32_t held[16];               // per tile, counted over all items, % 16: which of its pages hold tokens
  uint32_t tmem;
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    prompt_kernel(PromptParams P, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D>;
  constexpr int NT = C::kTiles, R = C::kRing, CB = D / 64, kPh = C::kPhases;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + NT * C::kQ;
  Small<D>& sm = *reinterpret_cast<Small<D>*>(ring + R * C::kKv);
  const AttnLaunch& p = P.a;
  const KvDev& kv = p.cache;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < R; ++i) {
      tc::mbar_init(&sm.full[i], 1);
      tc::mbar_init(&sm.empty[i], 2);  // the products and the warp that looks after V tiles
    }
    for (int i = 0; i < kPh; ++i) tc::mbar_init(&sm.checked[i], 1);
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&sm.s_ready[i >> 1][i & 1], 1);
      tc::mbar_init(&sm.p_ready[i >> 1][i & 1], 128);
      tc::mbar_init(&sm.pv_done[i >> 1][i & 1], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.q_ready[i], 128);
      tc::mbar_init(&sm.drain[i], 1);
    }
    tc::mbar_init_fence();
    tc::prefetch_map(&kmap);
    tc::prefetch_map(&vmap);
  }
  if (warp == 4 * NT) tc::tmem_alloc(&sm.tmem, 512);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Plan plan = plan_of(count_items<C::kRows, C::kThreads>(p, sm.sum), P.max_pieces);
  const uint32_t tmem = sm.tmem;
  const int ps = kv.page_size, shift = __ffs(ps) - 1, box = min(ps, kTN), boxes = kTN / box;
  const int bshift = __ffs(box) - 1;

  Finder<D> finder(p);
  Item w;
  bool ok = true;
  uint32_t at = 0;     // K and V tiles gone by; a K tile is entry at % R of the ring, its V tile the next
  uint32_t tiles = 0;  // cached tiles gone by
  const int role = warp - 4 * NT;  // < 0: softmax

  // (384 threads of one CTA an SM may take 168 registers each; the softmax, which holds a row of scores, sets the
  // kernel's 153 at d = 128.)
  if (role < 0) {
    // ---- softmax: a thread per query ----
    const int tile = warp >> 2, row = tid & 127;
    const float sl2 = p.scale * 1.4426950408889634f;
    uint8_t* qt = smem + tile * C::kQ;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t o_col = lane_base + C::kO + tile * D;
    uint32_t chk = 0;      // parity of checked, a bit per ring phase
    int64_t out_at = -1;   // of this thread's query; -1: none
    // Finds the item of a round and brings its queries to shared memory.  (No product reads those of the item
    // before any more once its last scores are ready.)
    auto begin = [&](int round) {
      if (!finder.find(plan, round, blockIdx.x, w)) return false;
      const int qi = w.q0 + tile * 128 + row;
      const bool mine = qi < w.r.len * p.G;
      int g = -1;
      if (mine) g = kv_token(p.rows, w.r.bos + qi / p.G, p.num_global, p.status);
      const int64_t head = (int64_t)(w.h * p.G + (mine ? qi % p.G : 0)) * D;
      out_at = g >= 0 ? (int64_t)g * p.out_stride + head : -1;
      load_queries<D>(p, qt, 32 * (warp & 3), g >= 0 ? (int64_t)g * p.q_stride + head : -1);
      tc::fence_async_smem();
      tc::mbar_arrive(&sm.q_ready[tile]);
      return true;
    };
    bool more = begin(0);
    for (int round = 0; more && ok; ++round) {
      const int qi = w.q0 + tile * 128 + row, nq = w.r.len * p.G;
      const int first = w.r.kv - w.r.len;  // position of the first new token
      const int pos = min(first + qi / p.G, w.r.kv - 1);
      const int tmin = first + min(w.q0 + tile * 128, nq - 1) / p.G, cmin = first + w.q0 / p.G;
      const int tmax = min(first + (w.q0 + tile * 128 + 127) / p.G, w.r.kv - 1);
      float m = -INFINITY, l = 0.f;  // the maximum that the weights refer to (of scores before their scale); their
                                     // sum, both pieces' and O's 2^-kGrow of e^(s - m)'s, which the join takes as it is
      bool wrote = false;            // O holds something, or will
      for (int j = w.j0; j < w.j1; ++j, ++tiles) {
        const uint32_t buf = tiles & 1, phase = tiles % kPh;
        const uint32_t s_col = lane_base + tile * 128 + buf * 64;
        const int b = tile_at(w, j);
        // O is complete when the product of the tile before is.  (The product two tiles before came before these
        // scores, so no phase can be taken for another.)
        auto o_complete = [&]() {
          const uint32_t last = tiles - 1;
          ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&sm.pv_done[tile][buf ^ 1], (last >> 1) & 1, P.wait_ns));
          tc::fence_after();
          return ok;
        };
        ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&sm.s_ready[tile][buf], (tiles >> 1) & 1, P.wait_ns));
        if (!ok) break;
        tc::fence_after();
        uint32_t r[2][32];
        ld_begin(s_col, r[0]);
        ld_begin(s_col + 32, r[1]);
        const uint32_t have = sm.held[tiles & 15];
        const bool all_pages = have == (1u << boxes) - 1u;
        const bool part = !all_pages || in_part(p, b, tmin, tmax);
        const bool look = in_part(p, b, cmin, w.last);
        ld_wait(r[0]);
        ld_wait(r[1]);
        if (part) {
          uint32_t vis[2];
          visible(p, b, pos, have, all_pages, bshift, vis);
          hide(r[0], vis[0]);
          hide(r[1], vis[1]);
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 32; ++i) m4[i & 3] = max3(m4[i & 3], __uint_as_float(r[0][i]), __uint_as_float(r[1][i]));
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        const bool grow = mx > m && (m == -INFINITY || (mx - m) * sl2 > kGrow);
        if (__any_sync(0xffffffffu, grow)) {
          const bool from = grow && m != -INFINITY;
          const float f = from ? ex2((m - mx) * sl2) : 1.f;
          if (grow) m = mx;
          l *= f;
          if (wrote && __any_sync(0xffffffffu, from)) {
            if (!o_complete()) break;
            scale_o<D>(o_col, f);
          }
        }
        const float ms = m == -INFINITY ? 0.f : fmaf(-m, sl2, -kGrow);  // so that the largest weight is 1
        const uint64_t scale = pair(sl2, sl2), shift = pair(ms, ms);
        uint64_t sum[2] = {0, 0};
        float u[32];
        weights32(r[0], scale, shift, sum, u);
        weights32(r[1], scale, shift, sum, u + 16);
        tc::tmem_st32(s_col, u);
        {
          float a0, a1;
          unpair(add2(sum[0], sum[1]), a0, a1);
          l += a0 + a1;
        }
        tc::tmem_st_wait();
        if (look) {
          ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&sm.checked[phase], (chk >> phase) & 1, P.wait_ns));
          chk ^= 1u << phase;
          if (!ok) break;
          if ((sm.bad[phase][0] | sm.bad[phase][1]) != 0) {
            if (wrote) {
              if (!o_complete()) break;
            } else {
              clear_o<D>(o_col);
            }
            add_listed<D>(p, w.r.trow, w.h, sm.bad[phase], b, pos, s_col, o_col);
          }
        }
        tc::fence_before();
        tc::mbar_arrive(&sm.p_ready[tile][buf]);
        wrote = true;
      }
      if (!ok) break;
      const bool cut = w.pieces > 1;
      const int64_t at = out_at;
      more = begin(round + 1);  // its first scores come up while O goes out
      if (wrote) {
        const uint32_t last = tiles - 1;
        ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&sm.pv_done[tile][last & 1], (last >> 1) & 1, P.wait_ns));
        if (!ok) break;
        tc::fence_after();
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t part_row = (int64_t)blockIdx.x * C::kRows + tile * 128 + row;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + max(at, (int64_t)0);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        if (wrote) {
          tc::tmem_ld32(o_col + c, o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
        if (cut) {
          float4* dst = reinterpret_cast<float4*>(P.part + part_row * D + c);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else if (at >= 0) {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= inv;
#pragma unroll
          for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(out + c + 8 * i) = tc::pack8(o + 8 * i);
        }
      }
      if (cut) *reinterpret_cast<float2*>(P.stats + part_row * 2) = make_float2(m, l);
    }
    if (!ok) set_status(p.status, GDN_STATUS_WAIT_TIMEOUT);
  } else if (role <= 1) {
    // ---- products: a lane of warp 0 issues all S = Q K^T, one of warp 1 all O += P V ----
    const uint32_t base = tc::smem_addr(smem);
    uint32_t chk = 0;  // parity of checked, a bit per ring phase
    // (a phase of a barrier; false once a wait has given up)
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && tc::mbar_wait(bar, parity & 1, P.wait_ns);
      if (ok) tc::fence_after();
      return ok;
    };
    // V of tile t, of this item's number j, is there; onto: O holds listed tokens' share by then
    auto v_ready = [&](uint32_t t, int j, int cmin, bool& onto) {
      const uint32_t phase = t % kPh;
      if (!wait(&sm.full[2 * phase + 1], t / kPh)) return false;
      if (!in_part(p, tile_at(w, j), cmin, w.last)) return true;
      if (!wait(&sm.checked[phase], chk >> phase)) return false;
      chk ^= 1u << phase;
      onto |= (sm.bad[phase][0] | sm.bad[phase][1]) != 0;
      return true;
    };
    for (int round = 0; round <= plan.full && ok; ++round) {
      if (!finder.find(plan, round, blockIdx.x, w)) break;
      const int n = w.j1 - w.j0, cmin = w.r.kv - w.r.len + w.q0 / p.G;
      if (lane == 0 && role == 0) {
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t t = tiles + j, buf = t & 1, phase = t % kPh;
          if (!wait(&sm.full[2 * phase], t / kPh)) break;
#pragma unroll
          for (uint32_t i = 0; i < NT; ++i) {
            if (j == 0 && !wait(&sm.q_ready[i], round)) break;
            // the buffer is free once the product two tiles before is done
            if (t >= 2 && !wait(&sm.pv_done[i][buf], (t >> 1) - 1)) break;
            s_products<D>(base, i, phase, i * 128 + buf * 64);
            tc::commit(&sm.s_ready[i][buf]);
          }
          tc::commit(&sm.empty[2 * phase]);
        }
      } else if (lane == 0) {
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t t = tiles + j, buf = t & 1, phase = t % kPh;
          bool onto = j > 0;
          if (!v_ready(t, w.j0 + j, cmin, onto)) break;
#pragma unroll
          for (uint32_t i = 0; i < NT; ++i) {
            if (!wait(&sm.p_ready[i][buf], t >> 1)) break;
            pv_products<D>(base, i, phase, i * 128 + buf * 64, onto);
            tc::commit(&sm.pv_done[i][buf]);
          }
          tc::commit(&sm.empty[2 * phase + 1]);
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      tiles += n;
    }
    if (lane == 0) {
      tc::commit(&sm.drain[role]);
      if (!tc::mbar_wait(&sm.drain[role], 0, P.wait_ns)) ok = false;
      if (!ok) set_status(p.status, GDN_STATUS_WAIT_TIMEOUT);
    }
    __syncwarp();
  } else if (role == 2) {
    // ---- fetches: a lane per page of the tile ----
    const int bi = lane, spp = slabs_per_page(kv);
    const int none = (kv.num_pages - 1) * spp + kv.Hkv;  // a slab past the pool
    const bool active = bi < boxes;
    uint32_t fetched = 0;  // tiles fetched, K and V
    for (int round = 0; round <= plan.full && ok; ++round) {
      if (!finder.find(plan, round, blockIdx.x, w)) break;
      const int32_t* row = kv.table + (int64_t)w.r.trow * kv.max_pages;
      const int entries = (w.r.kv + ps - 1) >> shift;
      int eb = -64, ids = 0, ahead = 0;  // 32 table entries are held, one per lane, and the 32 behind them
      for (int j = w.j0; j < w.j1 && ok; ++j, at += 2, ++tiles) {
        const int pos = tile_at(w, j) + bi * box, e = tile_at(w, j) >> shift;
        if (e >= eb + 32) {
          if (e < eb + 64) {
            ids = ahead;
            eb += 32;
          } else {
            eb = e;
            ids = eb + lane < entries ? load(row + eb + lane) : 0;
          }
          ahead = eb + 32 + lane < entries ? load(row + eb + 32 + lane) : 0;
        }
        int page = __shfl_sync(0xffffffffu, ids, active ? (pos >> shift) - eb : 0);
        page = active && pos < w.r.kv ? page_or_null(page, kv, p.status) : 0;
        const uint32_t mask = __ballot_sync(0xffffffffu, page > 0);
        for (int v = 0; v < 2; ++v) {
          const uint32_t a = at + v, en = a % R;
          ok = __all_sync(0xffffffffu, a < R || tc::mbar_wait(&sm.empty[en], (a / R - 1) & 1, P.wait_ns));
          if (!ok) break;
          if (lane == 0) {
            if (v == 0) sm.held[tiles & 15] = mask;
            tc::expect_tx(&sm.full[en], C::kKv);
          }
          __syncwarp();
          if (active)
            tc::tma_page(ring + en * C::kKv + bi * box * D * 2, v ? &vmap : &kmap, pos & (ps - 1),
                         page > 0 ? page * spp + w.h : none, &sm.full[en]);
          fetched = a + 1;
        }
        if (!ok) break;
      }
    }
    // No copy may be in flight when the CTA ends (the products wait for every tile, so this passes at
    // once unless a wait gave up).
    for (uint32_t a = fetched > (uint32_t)R ? fetched - R : 0; a < fetched; ++a)
      ok &= tc::mbar_wait(&sm.full[a % R], (a / R) & 1, P.wait_ns);
    if (!ok) set_status(p.status, GDN_STATUS_WAIT_TIMEOUT);
  } else {
    // ---- V tiles that some query sees in part ----
    // (this warp goes through every V tile, so that no phase is taken for another)
    for (int round = 0; round <= plan.full && ok; ++round) {
      if (!finder.find(plan, round, blockIdx.x, w)) break;
      const int cmin = w.r.kv - w.r.len + w.q0 / p.G;
      for (int j = w.j0; j < w.j1 && ok; ++j, at += 2) {
        const int b = tile_at(w, j);
        const uint32_t en = (at + 1) % R;
        const bool look = in_part(p, b, cmin, w.last);
        for (int v = 0; v < 2; ++v) {
          const uint32_t a = at + v;
          ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&sm.full[a % R], (a / R) & 1, P.wait_ns));
          if (!ok) break;
          if (lane == 0 && (v == 0 || !look)) tc::mbar_arrive(&sm.empty[a % R]);
        }
        if (!ok || !look) continue;
#pragma unroll 1
        for (int u = 0; u < kTN / 32; ++u) {
          const int t = u * 32 + lane;
          uint8_t* v = ring + en * C::kKv + (t >> 3) * CB * 1024 + (t & 7) * 128;
          uint32_t acc[4] = {0, 0, 0, 0};
          const bool past = b + t >= w.r.kv;
#pragma unroll 8
          for (int c = 0; c < D / 8; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(v + (c >> 3) * 1024 + (((c & 7) ^ (t & 7)) << 4));
            acc[0] = note2(x.x, acc[0]);
            acc[1] = note2(x.y, acc[1]);
            acc[2] = note2(x.z, acc[2]);
            acc[3] = note2(x.w, acc[3]);
          }
          const bool odd = ((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7fff7fffu) != 0;
          if (past || odd)
            for (int c = 0; c < D / 8; ++c)
              *reinterpret_cast<uint4*>(v + (c >> 3) * 1024 + (((c & 7) ^ (t & 7)) << 4)) = make_uint4(0, 0, 0, 0);
          const uint32_t list = __ballot_sync(0xffffffffu, odd && !past);
          if (lane == 0) sm.bad[en >> 1][u] = list;
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(&sm.checked[en >> 1]);
          tc::mbar_arrive(&sm.empty[en]);
        }
      }
    }
    if (!ok) set_status(p.status, GDN_STATUS_WAIT_TIMEOUT);
  }
  tc::fence_before();
  __syncthreads();
  if (role == 0) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Adds the pieces of an item's queries in order: a warp per query, kJoinRows queries per block, four pieces' values on
// their way at a time.
constexpr int kJoinRows = 8;
template <int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(PromptParams P) {
  constexpr int kRows = Cfg<D>::kRows, E = D / 32;
  __shared__ int64_t sum[8];
  const AttnLaunch& p = P.a;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Plan plan = plan_of(count_items<kRows, 256>(p, sum), P.max_pieces);
  const int pieces = plan.pieces;
  if (pieces == 1 || (int)blockIdx.x >= plan.left) return;
  Finder<D> finder(p);
  Item w;
  if (!finder.find(plan, plan.full, blockIdx.x * pieces, w)) return;
  const float sl2 = p.scale * 1.4426950408889634f;
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y * kJoinRows + (threadIdx.x >> 5);
  const int qi = w.q0 + r;
  if (qi >= w.r.len * p.G) return;
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.f;
  // lane s holds piece s's (m, l)
  const int64_t row0 = (int64_t)blockIdx.x * pieces * kRows + r;
  const float2 st = lane < pieces ? *reinterpret_cast<const float2*>(P.stats + (row0 + (int64_t)lane * kRows) * 2)
                                  : make_float2(-INFINITY, 0.f);
  m = st.x;
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float f = st.x == -INFINITY ? 0.f : ex2((st.x - m) * sl2);
  for (int s0 = 0; s0 < pieces; s0 += 4) {
    float x[4][E];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool there = __shfl_sync(0xffffffffu, st.x, s0 + u) != -INFINITY;  // (lanes past the pieces hold none)
#pragma unroll
      for (int i = 0; i < E; ++i)
        x[u][i] = there ? P.part[(row0 + (int64_t)(s0 + u) * kRows) * D + lane + 32 * i] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float fs = __shfl_sync(0xffffffffu, f, s0 + u);
      l += __shfl_sync(0xffffffffu, st.y, s0 + u) * fs;
#pragma unroll
      for (int i = 0; i < E; ++i) o[i] += x[u][i] * fs;
    }
  }
  const int t = qi / p.G;
  const int g = p.rows.tok ? load(p.rows.tok + w.r.bos + t) : w.r.bos + t;
  if (g < 0 || g >= p.num_global) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* out =
      static_cast<__nv_bfloat16*>(p.out) + (int64_t)g * p.out_stride + (int64_t)(w.h * p.G + qi - t * p.G) * D;
#pragma unroll
  for (int i = 0; i < E; ++i) out[lane + 32 * i] = __float2bfloat16_rn(o[i] * inv);
}

// The pieces that an item of the last round may be cut into: as the items of a single row say, any number when
// there are several rows, whose lengths the host does not know.
int max_pieces(const AttnLaunch& a, int rows) {
  if (a.rows.num_seqs > 1) return kMaxPieces;
  return plan_of(((int64_t)a.rows.num_tokens * a.G + rows - 1) / rows * a.cache.Hkv, kMaxPieces).pieces;
}

template <int D>
cudaError_t launch_d(const AttnLaunch& a, cudaStream_t s) {
  using C = Cfg<D>;
  static std::atomic<uint64_t> done{0};
  constexpr int smem = (int)(C::kSmem + sizeof(Small<D>));
  static_assert(smem <= 232448, "shared memory");
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap kmap, vmap;
  if (!encode_pool_maps(a.cache, a.cache.page_size < kTN ? a.cache.page_size : kTN, &kmap, &vmap))
    return cudaErrorInvalidValue;
  PromptParams P{};
  P.a = a;
  P.max_pieces = max_pieces(a, C::kRows);
  P.stats = static_cast<float*>(a.ws);
  P.part = P.stats + (size_t)2 * kSms * C::kRows;
  P.wait_ns = kDefaultWaitNs;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSms);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, prompt_kernel<D>, P, kmap, vmap)) != cudaSuccess || P.max_pieces == 1) return e;
  cfg.gridDim = dim3(kSms / 2, C::kRows / kJoinRows);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, prompt_join_kernel<D>, P);
}

}  // namespace

bool attn_prompt_supported(const AttnLaunch& a, gdn_dtype dtype) {
  const int d = a.cache.d;
  return dtype == GDN_BF16 && (d == 64 || d == 128 || d == 256);
}

size_t attn_prompt_workspace(const AttnLaunch& a) {
  const int d = a.cache.d, rows = d <= 128 ? 256 : 128;
  return max_pieces(a, rows) == 1 ? 0 : (size_t)kSms * rows * (d + 2) * 4;
}

cudaError_t launch_attn_prompt(const AttnLaunch& a, cudaStream_t s) {
  return a.cache.d == 64 ? launch_d<64>(a, s) : a.cache.d == 128 ? launch_d<128>(a, s) : launch_d<256>(a, s);
}

}  // namespace gdn
