// gdn_attn_split.cu -- attention of decode and verify rows over the paged cache (bf16, d = 64, 128, 256).
//
// Up to 64 queries (new tokens x q-heads of one kv-head) share every key and value, so the bytes of
// the cache bound the kernel: 4 flops per query per element against 2 bytes, far under the tensor
// cores' ratio.  What matters is that every SM streams its share of the cache without a pause.
//
// Work.  A unit is one (row, kv-head): the TN-token tiles that its queries see, window and first
// tokens included.  All units' tiles laid end to end are cut into equal shares, one per CTA, so
// ragged lengths and a single long row load the SMs alike.  A share's piece of a unit that is not the
// whole unit leaves (m, l, o) in the workspace; the join kernel adds a unit's pieces in the order of
// the CTAs, so results do not depend on timing.
//
// A CTA: one warp fetches pages by TMA into a ring of stages (up to 192 KB in flight; a NULL page is
// fetched from past the pool and reads as zeros) and the queries of the next unit; 4 or 8 warps
// compute, each 32 tokens of a tile against 16 queries with mma.m16n8k16 and a running maximum and
// sum of its own, and meet only where a unit ends.  The weights enter the second product as a bf16
// pair (hi + lo), so they keep 16 bits: the product is nearly free here, and one bf16 would cost as
// much accuracy as the output's own rounding.
#include "gdn_tma.cuh"

namespace gdn {

namespace {

constexpr int kSplitCtas = 152;  // one per SM
constexpr uint32_t kSmemBytes = 230400;  // dynamic, behind the alignment: ring, merge buffer, queries
constexpr int kJoinWarps = 8;

// WQ groups of 16 queries x DS slices of the values' columns x KG groups of 32 tokens, a warp each.
template <int D, int WQ, int DS, int KG>
struct Cfg {
  static constexpr int kWarps = WQ * DS * KG;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kTN = D == 256 ? 32 : 64;                    // tokens of a tile
  static constexpr int kKT = kTN / 32;                              // 32-token steps of a tile
  static constexpr int kTG = KG / kKT;                              // tiles worked on at a time
  static constexpr int kNQ = 16 * WQ;                               // queries of a unit, at most
  static constexpr int kDV = D / DS;                                // value columns of a warp
  static constexpr uint32_t kHalf = (uint32_t)kTN * D * 2;          // K (or V) bytes of a stage
  static constexpr int kSP = D == 64 && KG > 1 ? KG / 2 : 1;        // token groups that merge at a time
  static constexpr int kSlots = kSP * WQ * DS;                      // of the merge buffer, a warp's output each
  static constexpr uint32_t kMerge = (uint32_t)kSlots * 16 * kDV * 4;
  static constexpr uint32_t kPitch = D * 2 + 16;                    // bytes of a query: rows 16 bytes apart mod 128
  static constexpr uint32_t kQ = kNQ * kPitch;                      // one of two buffers
  static constexpr int kFit = (int)((kSmemBytes - kMerge - 2 * kQ) / (2 * kHalf));
  // A multiple of kTG: a stage is always worked on by the same warps, so none can miss a phase of its barrier.
  static constexpr int kStages = (kFit < 16 ? kFit : 16) / kTG * kTG;
  static constexpr uint32_t kRing = (uint32_t)kStages * 2 * kHalf;
  static_assert(kKT * kTG == KG && kStages > kTG, "ring too short");
  static_assert(kRing + kMerge + 2 * kQ <= kSmemBytes && kRing % 1024 == 0, "shared memory");
};

struct SplitParams {
  AttnLaunch a;
  float* part;     // [2 * kSplitCtas][kNQ][D]
  float* stats;    // [2 * kSplitCtas][kNQ][2]: m (log2 units), l
  int32_t* info;   // [kSplitCtas][8]: the unit that begins in a CTA and ends in another
  uint64_t wait_ns;
};

struct Unit {
  KvRow r;
  int sink_tiles, first_tile, tiles;
};

// The tiles that row n's queries see; 0 for an empty or bad row.
template <int TN>
__device__ __forceinline__ Unit unit_of(const AttnLaunch& p, int n, uint32_t* st) {
  Unit u;
  u.tiles = u.sink_tiles = u.first_tile = 0;
  if (!load_kv_row(p.rows, p.cache, n, u.r, st) || u.r.len == 0) return u;
  const int low = p.window > 0 ? max(0, u.r.kv - u.r.len - p.window + 1) : 0;
  u.sink_tiles = (min(p.sinks, low) + TN - 1) / TN;
  u.first_tile = max(low / TN, u.sink_tiles);
  u.tiles = u.sink_tiles + (u.r.kv + TN - 1) / TN - u.first_tile;
  return u;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// Whether one of the two bf16 of x is an infinity or NaN.
__device__ __forceinline__ bool not_finite2(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}
template <int WARPS>
__device__ __forceinline__ void compute_bar() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * WARPS) : "memory");
}

// The CTA's share of all tiles, and where it begins.
struct Share {
  int64_t total, first, last;
  int row;
  int64_t into;  // tiles of row `row` before the share
};

template <int TN, int THREADS>
__device__ void find_share(const AttnLaunch& p, int ctas, int cta, Share& out) {
  __shared__ int64_t s_part[THREADS / 32];
  __shared__ Share s_share;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.rows.num_seqs + THREADS - 1) / THREADS;
  const int n0 = min(tid * per, p.rows.num_seqs), n1 = min(n0 + per, p.rows.num_seqs);
  int64_t mine = 0;
  for (int n = n0; n < n1; ++n) mine += unit_of<TN>(p, n, cta == 0 ? p.status : nullptr).tiles;
  mine *= p.cache.Hkv;
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s_part[warp] = inc;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) before += s_part[i];
    total += s_part[i];
  }
  before += inc - mine;
  const int64_t used = min((int64_t)ctas, total);  // a share holds a tile at least
  int64_t first = total, last = total;
  if (cta < used) {
    first = total * cta / used;
    last = total * (cta + 1) / used;
  }
  if (tid == 0) {
    s_share.total = total;
    s_share.first = first;
    s_share.last = last;
    s_share.row = 0;
    s_share.into = 0;
  }
  __syncthreads();
  if (first < last && first >= before && first < before + mine) {  // one thread
    int64_t at = before;
    for (int n = n0; n < n1; ++n) {
      const int64_t t = (int64_t)unit_of<TN>(p, n, nullptr).tiles * p.cache.Hkv;
      if (first < at + t) {
        s_share.row = n;
        s_share.into = first - at;
        break;
      }
      at += t;
    }
  }
  __syncthreads();
  out = s_share;
}

// Walks the units of a share: (row, head, tiles [j0, j0 + len) of the unit).  A warp holds 32 rows,
// one per lane, so that going on to the next row waits for no memory.  All lanes call together.
template <int TN>
struct Walk {
  const AttnLaunch& p;
  int64_t left;
  int n, h, j0, len;
  Unit u;
  __device__ Walk(const AttnLaunch& launch, const Share& s) : p(launch), left(s.last - s.first), n(s.row), len(0) {
    if (left <= 0) return;
    fill();
    pick();
    h = (int)(s.into / u.tiles);
    j0 = (int)(s.into - (int64_t)h * u.tiles);
    len = (int)min((int64_t)(u.tiles - j0), left);
  }
  __device__ bool valid() const { return left > 0; }
  __device__ void next() {
    left -= len;
    if (left <= 0) return;
    j0 = 0;
    if (++h == p.cache.Hkv) {
      h = 0;
      do {
        if (++n >= p.rows.num_seqs) {
          left = 0;
          return;
        }
        if (n == base + 32) fill();
        pick();
      } while (u.tiles == 0);
    }
    len = (int)min((int64_t)u.tiles, left);
  }
  __device__ int tile_at(int j) const { return (j < u.sink_tiles ? j : u.first_tile + j - u.sink_tiles) * TN; }

 private:
  int base;
  Unit mine;
  __device__ void fill() {
    base = n;
    mine.tiles = 0;
    const int row = n + (threadIdx.x & 31);
    if (row < p.rows.num_seqs) mine = unit_of<TN>(p, row, nullptr);
  }
  __device__ void pick() {
    const int src = n - base;
    u.r.bos = __shfl_sync(0xffffffffu, mine.r.bos, src);
    u.r.len = __shfl_sync(0xffffffffu, mine.r.len, src);
    u.r.kv = __shfl_sync(0xffffffffu, mine.r.kv, src);
    u.r.trow = __shfl_sync(0xffffffffu, mine.r.trow, src);
    u.sink_tiles = __shfl_sync(0xffffffffu, mine.sink_tiles, src);
    u.first_tile = __shfl_sync(0xffffffffu, mine.first_tile, src);
    u.tiles = __shfl_sync(0xffffffffu, mine.tiles, src);
  }
};

// One 32-token step's second product, O += P V.  PART: some query does not see some token, so the
// values must not reach it whatever they hold.
template <bool PART, int TN, int DV>
__device__ __forceinline__ void values_step(float (&o)[DV / 8][4], const uint32_t (&ph)[2][4], const uint32_t (&pl)[2][4],
                                            uint32_t vbase, int col0, int b, const int (&pos)[2], int pmax, int window,
                                            int sinks) {
  const int lane = threadIdx.x & 31, c2 = (lane & 3) * 2;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    // lanes 0-7, 8-15, 16-23, 24-31 point at (tokens 0-7, left 8 columns), (8-15, left), (0-7, right),
    // (8-15, right); the transposing load puts two tokens of a column into a register
    const int r = (lane & 7) + (((lane >> 3) & 1) << 3);
    const uint32_t base = vbase + (half * 16 + r) * 128;
    const int t0 = b + half * 16;
    uint32_t m0 = 0xffffffffu, m1 = 0xffffffffu;
    if (PART) {  // tokens past the row's end hold anything
      m0 = (t0 + c2 <= pmax ? 0xffffu : 0u) | (t0 + c2 + 1 <= pmax ? 0xffff0000u : 0u);
      m1 = (t0 + c2 + 8 <= pmax ? 0xffffu : 0u) | (t0 + c2 + 9 <= pmax ? 0xffff0000u : 0u);
    }
#pragma unroll
    for (int i = 0; i < DV / 16; ++i) {
      const int chunk = col0 / 8 + i * 2 + (lane >> 4);
      uint32_t v[4];
      ldsm4t(v, base + (chunk >> 3) * TN * 128 + (((chunk & 7) ^ (r & 7)) << 4));
      if (PART) {
        v[0] &= m0;
        v[1] &= m1;
        v[2] &= m0;
        v[3] &= m1;
        const bool odd = not_finite2(v[0]) || not_finite2(v[1]) || not_finite2(v[2]) || not_finite2(v[3]);
        if (__any_sync(0xffffffffu, odd)) {
          // An infinity or NaN that some query of the step must not see (0 times it is NaN): one token
          // at a time, added only where it is seen.
#pragma unroll 1
          for (int t = 0; t < 16; ++t) {
            const uint32_t keep = ((t & 7) >> 1) == (lane & 3) ? ((t & 1) ? 0xffff0000u : 0xffffu) : 0u;
            const uint32_t lo = t < 8 ? keep : 0u, hi = t < 8 ? 0u : keep;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              float x[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816(x, ph[half], v[2 * n] & lo, v[2 * n + 1] & hi);
              mma16816(x, pl[half], v[2 * n] & lo, v[2 * n + 1] & hi);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int at = pos[e >> 1], tk = t0 + t;
                if (tk <= at && (window <= 0 || tk > at - window || tk < sinks)) o[2 * i + n][e] += x[e];
              }
            }
          }
          continue;
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        mma16816(o[2 * i + n], ph[half], v[2 * n], v[2 * n + 1]);
        mma16816(o[2 * i + n], pl[half], v[2 * n], v[2 * n + 1]);
      }
    }
  }
}

template <int D, int WQ, int DS, int KG>
__global__ void __launch_bounds__(Cfg<D, WQ, DS, KG>::kThreads, 1)
    split_kernel(SplitParams P, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D, WQ, DS, KG>;
  constexpr int TN = C::kTN, S = C::kStages, DV = C::kDV;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  float* merge = reinterpret_cast<float*>(ring + C::kRing);
  uint8_t* qbuf = ring + C::kRing + C::kMerge;
  __shared__ uint64_t full[S], empty[S], qfull[2], qempty[2];
  __shared__ uint32_t held[S];  // per stage: which of the tile's pages hold tokens
  __shared__ float sm_m[C::kSlots][16], sm_l[C::kSlots][16];
  __shared__ int dead;
  const AttnLaunch& p = P.a;
  const KvDev& kv = p.cache;
  // The warp's number comes from a shuffle, so that the compiler takes it as one value of the warp and
  // infers no range for it: with threadIdx.x / 32 nvcc 13.0 took the receiving groups' slots of the
  // merge buffer below to lie outside it.
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], C::kKT * WQ * DS);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&qfull[i], 1);
      tc::mbar_init(&qempty[i], C::kWarps);
    }
    tc::mbar_init_fence();
    dead = 0;
    P.info[blockIdx.x * 8] = 0;
  }
  if (tid == 32 * C::kWarps) {
    tc::prefetch_map(&kmap);
    tc::prefetch_map(&vmap);
  }
  Share share;
  find_share<TN, C::kThreads>(p, kSplitCtas, blockIdx.x, share);
  const int ps = kv.page_size;
  const int box = min(ps, TN);       // tokens of one copy
  const int boxes = TN / box;        // pages of a tile
  const int shift = __ffs(ps) - 1;

  if (warp == C::kWarps) {
    // ---- the fetching warp: lane = (page of the tile, 64-column block, K or V) ----
    constexpr int CB = D / 64;
    const int bi = lane / (2 * CB), cb = (lane >> 1) % CB, is_v = lane & 1;
    const bool active = bi < boxes;
    int it = 0, seg = 0;
    bool ok = true;
    for (Walk<TN> w(p, share); w.valid() && ok; w.next(), ++seg) {
      // the unit's queries
      const int nq = w.u.r.len * p.G, qb = seg & 1;
      int g[2];
      int rows = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int qi = lane + 32 * u;
        g[u] = -1;
        if (qi < nq) g[u] = global_token(RowsDev{nullptr, p.rows.tok}, w.u.r.bos + qi / p.G, p.num_global, p.status);
        rows += __popc(__ballot_sync(0xffffffffu, g[u] >= 0));
      }
      ok = seg < 2 || tc::mbar_wait(&qempty[qb], ((seg >> 1) - 1) & 1, P.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) tc::expect_tx(&qfull[qb], (uint32_t)rows * D * 2);
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int qi = lane + 32 * u;
        if (g[u] >= 0)
          tc::bulk_g2s(qbuf + qb * C::kQ + qi * C::kPitch,
                       static_cast<const __nv_bfloat16*>(p.q) + (int64_t)g[u] * p.q_stride +
                           (int64_t)(w.h * p.G + qi % p.G) * D,
                       D * 2, &qfull[qb]);
      }
      // 32 table entries are held, one per lane, and the 32 behind them are on their way
      const int32_t* row = kv.table + (int64_t)w.u.r.trow * kv.max_pages;
      const int entries = (w.u.r.kv + ps - 1) >> shift;
      int eb = -64, ids = 0, ahead = 0;
      for (int j = w.j0; j < w.j0 + w.len; ++j, ++it) {
        const int pos = w.tile_at(j) + bi * box;
        const int e = w.tile_at(j) >> shift;
        if (e >= eb + 32) {
          if (e < eb + 64) {
            ids = ahead;
            eb += 32;
          } else {
            eb = e;
            ids = eb + lane < entries ? __ldg(row + eb + lane) : 0;
          }
          ahead = eb + 32 + lane < entries ? __ldg(row + eb + 32 + lane) : 0;
        }
        int page = __shfl_sync(0xffffffffu, ids, active ? (pos >> shift) - eb : 0);
        page = active && pos < w.u.r.kv ? page_or_null(page, kv, p.status) : 0;
        const int s = it % S;
        ok = it < S || tc::mbar_wait(&empty[s], ((it / S) - 1) & 1, P.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t have = __ballot_sync(0xffffffffu, page > 0 && cb == 0 && is_v == 0);
        uint32_t mask = 0;
        for (int i = 0; i < boxes; ++i) mask |= (have >> (i * 2 * CB) & 1u) << i;
        if (lane == 0) {
          held[s] = mask;
          tc::expect_tx(&full[s], 2 * C::kHalf);
        }
        __syncwarp();
        if (active) {
          uint8_t* dst = ring + (size_t)s * 2 * C::kHalf + is_v * C::kHalf + (size_t)(cb * TN + bi * box) * 128;
          tc::tma_page(dst, is_v ? &vmap : &kmap, cb * 64, pos & (ps - 1), w.h, page > 0 ? page : kv.num_pages,
                       &full[s]);
        }
      }
    }
    // No copy may be in flight when the CTA ends.  Computing warps wait for every stage they use, so
    // this passes at once unless a wait gave up.
    for (int i = max(0, it - S); i < it; ++i) ok &= tc::mbar_wait(&full[i % S], (i / S) & 1, P.wait_ns);
    for (int i = max(0, seg - 2); i < seg; ++i) ok &= tc::mbar_wait(&qfull[i & 1], (i >> 1) & 1, P.wait_ns);
    if (!ok && lane == 0) {
      dead = 1;
      set_status(p.status, GDN_STATUS_WAIT_TIMEOUT);
    }
    return;
  }

  // ---- computing warps ----
  const int ds = warp % DS, wq = (warp / DS) % WQ, kg = warp / (DS * WQ);
  const int kt = kg % C::kKT, tg = kg / C::kKT;
  const int r8 = lane >> 2, c2 = (lane & 3) * 2;
  const int bshift = __ffs(box) - 1;
  const float sl2 = p.scale * 1.4426950408889634f;
  int it = 0, seg = 0;
  bool ok = true;
  for (Walk<TN> w(p, share); w.valid(); w.next(), ++seg) {
    const KvRow row = w.u.r;
    const int nq = row.len * p.G;
    const int pmin = row.kv - row.len, pmax = row.kv - 1;
    float o[DV / 8][4], m[2], l[2];
    int pos[2];  // the positions of this thread's two queries, r8 and r8 + 8 of the group's 16
#pragma unroll
    for (int i = 0; i < DV / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[e] = -INFINITY;
      l[e] = 0.f;
      pos[e] = min(pmin + (wq * 16 + r8 + 8 * e) / p.G, pmax);
    }
    ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&qfull[seg & 1], (seg >> 1) & 1, P.wait_ns));
    const uint32_t qbase =
        tc::smem_addr(qbuf + (seg & 1) * C::kQ) + (wq * 16 + (lane & 15)) * C::kPitch + (lane >> 4) * 16;

    for (int j = w.j0; j < w.j0 + w.len; ++j, ++it) {
      if (C::kTG > 1 && it % C::kTG != tg) continue;
      const int s = it % S;
      ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&full[s], (it / S) & 1, P.wait_ns));
      const int b = w.tile_at(j) + kt * 32;  // first token of this warp's step
      // a page is 16 tokens or more: the step's two halves may differ in whether theirs is NULL
      const uint32_t hm = held[s];
      const bool have0 = hm >> (kt * 32 >> bshift) & 1u, have1 = hm >> ((kt * 32 + 16) >> bshift) & 1u;
      if (ok && b <= pmax && (have0 || have1)) {
        const uint32_t kbase = tc::smem_addr(ring + (size_t)s * 2 * C::kHalf) + kt * 32 * 128;
        const uint32_t vbase = kbase + C::kHalf;
        // S = Q K^T.  K as the B operand: lanes 0-7, 8-15, 16-23, 24-31 point at (tokens 0-7, left 8
        // columns), (0-7, right), (8-15, left), (8-15, right) of 16 tokens.
        float sc[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
        {
          const int r = (lane & 7) + ((lane >> 4) << 3);
          const uint32_t base = kbase + r * 128;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t a[4], k0[4], k1[4];
            const uint32_t at =
                base + (k >> 2) * TN * 128 + ((((k & 3) * 2 + ((lane >> 3) & 1)) ^ (r & 7)) << 4);
            ldsm4(a, qbase + k * 32);
            ldsm4(k0, at);
            ldsm4(k1, at + 16 * 128);
            mma16816(sc[0], a, k0[0], k0[1]);
            mma16816(sc[1], a, k0[2], k0[3]);
            mma16816(sc[2], a, k1[0], k1[1]);
            mma16816(sc[3], a, k1[2], k1[3]);
          }
        }
        // not every query sees every token?
        const bool part = b + 31 > pmin || !have0 || !have1 ||
                          (p.window > 0 && b <= pmax - p.window && b + 31 >= p.sinks);
        if (part) {
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tok = b + n * 8 + c2 + (e & 1), at = pos[e >> 1];
              const bool sees = tok <= at && (p.window <= 0 || tok > at - p.window || tok < p.sinks) &&
                                (n < 2 ? have0 : have1);
              if (!sees) sc[n][e] = -INFINITY;
            }
        }
        // running maximum (of the raw scores; scale > 0), sum and output
        float mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = m[e];
#pragma unroll
          for (int n = 0; n < 4; ++n) x = fmaxf(x, fmaxf(sc[n][2 * e], sc[n][2 * e + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          mx[e] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f[e] = m[e] == -INFINITY ? 0.f : ex2((m[e] - mx[e]) * sl2);
            m[e] = mx[e];
            l[e] *= f[e];
          }
#pragma unroll
          for (int i = 0; i < DV / 8; ++i) {
            o[i][0] *= f[0];
            o[i][1] *= f[0];
            o[i][2] *= f[1];
            o[i][3] *= f[1];
          }
        }
        // P as the A operand: the score fragments are already in its layout
        uint32_t ph[2][4], pl[2][4];
        float ms[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) ms[e] = m[e] == -INFINITY ? 0.f : -m[e] * sl2;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          float e4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) e4[e] = ex2(fmaf(sc[n][e], sl2, ms[e >> 1]));
          l[0] += e4[0] + e4[1];
          l[1] += e4[2] + e4[3];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t hi = pack2(e4[2 * hf], e4[2 * hf + 1]);
            ph[n >> 1][(n & 1) * 2 + hf] = hi;
            pl[n >> 1][(n & 1) * 2 + hf] = pack2(e4[2 * hf] - bf_lo(hi), e4[2 * hf + 1] - bf_hi(hi));
          }
        }
        if (part)
          values_step<true, TN, DV>(o, ph, pl, vbase, ds * DV, b, pos, pmax, p.window, p.sinks);
        else
          values_step<false, TN, DV>(o, ph, pl, vbase, ds * DV, b, pos, pmax, p.window, p.sinks);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty[s]);
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&qempty[seg & 1]);

    // ---- the unit's piece ends: join the warps of a query group and column slice ----
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }
    if (!ok && lane == 0) {
      dead = 1;
      set_status(p.status, GDN_STATUS_WAIT_TIMEOUT);
    }
    // token groups hand theirs down, kSP of them at a time, through the merge buffer: the upper ones
    // give, the ones just below them receive, until group 0 holds all
#pragma unroll 1
    for (int live = KG; live > 1;) {
      const int take = min(live >> 1, C::kSP);
      const int gives = kg - (live - take), receives = gives + take;
      compute_bar<C::kWarps>();
      if (gives >= 0 && gives < take) {
        const int slot = (gives * WQ + wq) * DS + ds;
        float4* b4 = reinterpret_cast<float4*>(merge) + slot * (DV / 8) * 32 + lane;
#pragma unroll
        for (int i = 0; i < DV / 8; ++i) b4[i * 32] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        if ((lane & 3) == 0)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            sm_m[slot][r8 + 8 * e] = m[e];
            sm_l[slot][r8 + 8 * e] = l[e];
          }
      }
      compute_bar<C::kWarps>();
      if (receives >= 0 && receives < take) {
        const int slot = (receives * WQ + wq) * DS + ds;
        const float4* b4 = reinterpret_cast<const float4*>(merge) + slot * (DV / 8) * 32 + lane;
        float f[2], g[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float m2 = sm_m[slot][r8 + 8 * e], mn = fmaxf(m[e], m2);
          f[e] = m[e] == -INFINITY ? 0.f : ex2((m[e] - mn) * sl2);
          g[e] = m2 == -INFINITY ? 0.f : ex2((m2 - mn) * sl2);
          l[e] = l[e] * f[e] + sm_l[slot][r8 + 8 * e] * g[e];
          m[e] = mn;
        }
#pragma unroll
        for (int i = 0; i < DV / 8; ++i) {
          const float4 v = b4[i * 32];
          o[i][0] = o[i][0] * f[0] + v.x * g[0];
          o[i][1] = o[i][1] * f[0] + v.y * g[0];
          o[i][2] = o[i][2] * f[1] + v.z * g[1];
          o[i][3] = o[i][3] * f[1] + v.w * g[1];
        }
      }
      live -= take;
    }
    compute_bar<C::kWarps>();
    if (kg == 0 && !*(volatile int*)&dead) {
      const bool whole = w.j0 == 0 && w.len == w.u.tiles;
      // rows of queries in shared memory, then 16-byte stores
      float* mine = merge + (size_t)(wq * DS + ds) * 16 * DV;
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) f[e] = !whole ? 1.f : l[e] == 0.f ? 0.f : 1.f / l[e];
#pragma unroll
      for (int i = 0; i < DV / 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float2*>(mine + (r8 + 8 * e) * DV + i * 8 + c2) =
              make_float2(o[i][2 * e] * f[e], o[i][2 * e + 1] * f[e]);
      __syncwarp();
      if (whole) {
#pragma unroll 1
        for (int v = lane; v < 16 * DV / 8; v += 32) {
          const int q = v / (DV / 8), d0 = (v % (DV / 8)) * 8, qi = wq * 16 + q;
          if (qi >= nq) continue;
          const int t = qi / p.G;
          const int g = p.rows.tok ? __ldg(p.rows.tok + row.bos + t) : row.bos + t;
          if (g < 0 || g >= p.num_global) continue;
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + (int64_t)g * p.out_stride +
                                    (int64_t)(w.h * p.G + qi - t * p.G) * D + ds * DV + d0) =
              tc::pack8(mine + q * DV + d0);
        }
      } else {
        const int slot = 2 * blockIdx.x + (w.j0 == 0 ? 1 : 0);
#pragma unroll 1
        for (int v = lane; v < 16 * DV / 4; v += 32) {
          const int q = v / (DV / 4), d0 = (v % (DV / 4)) * 4;
          if (wq * 16 + q < nq)
            *reinterpret_cast<float4*>(P.part + ((size_t)slot * C::kNQ + wq * 16 + q) * D + ds * DV + d0) =
                *reinterpret_cast<const float4*>(mine + q * DV + d0);
        }
        if (ds == 0 && (lane & 3) == 0)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* st = P.stats + ((size_t)slot * C::kNQ + wq * 16 + r8 + 8 * e) * 2;
            st[0] = m[e];
            st[1] = l[e];
          }
        if (w.j0 == 0 && tid == 0) {
          // the CTA that holds the unit's last tile
          const int64_t used = min((int64_t)kSplitCtas, share.total);
          const int64_t end = share.last - w.left + w.u.tiles - 1;
          int32_t* info = P.info + blockIdx.x * 8;
          info[1] = row.bos;
          info[2] = nq;
          info[3] = w.h;
          info[4] = (int)(((end + 1) * used - 1) / share.total);
          info[0] = 1;
        }
      }
    }
  }
}

// Adds the pieces of the unit that begins in CTA blockIdx.x and ends in a later one; a block per
// query, its warps over the pieces.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(SplitParams P, int queries) {
  const float sl2 = P.a.scale * 1.4426950408889634f;
  __shared__ float so[kJoinWarps][D];
  __shared__ float sl[kJoinWarps], sm[kJoinWarps];
  const AttnLaunch& p = P.a;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c0 = blockIdx.x, qi = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t* info = P.info + c0 * 8;
  if (!info[0] || qi >= info[2]) return;
  const int bos = info[1], h = info[3], c1 = info[4];
  constexpr int E = D / 32;
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.f;
  for (int c = c0 + warp; c <= c1; c += kJoinWarps) {
    const size_t at = (size_t)(2 * c + (c == c0 ? 1 : 0)) * queries + qi;
    const float m2 = P.stats[at * 2], l2 = P.stats[at * 2 + 1];
    float v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = P.part[at * D + lane + 32 * i];
    const float mn = fmaxf(m, m2);
    const float a = m == -INFINITY ? 0.f : ex2((m - mn) * sl2), b = m2 == -INFINITY ? 0.f : ex2((m2 - mn) * sl2);
    l = l * a + l2 * b;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * a + v[i] * b;
    m = mn;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) so[warp][lane + 32 * i] = o[i];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float M = sm[0];
#pragma unroll
  for (int i = 1; i < kJoinWarps; ++i) M = fmaxf(M, sm[i]);
  float L = 0.f, f[kJoinWarps];
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) {
    f[i] = sm[i] == -INFINITY ? 0.f : ex2((sm[i] - M) * sl2);
    L += sl[i] * f[i];
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int t = qi / p.G;
  const int g = p.rows.tok ? __ldg(p.rows.tok + bos + t) : bos + t;
  if (g < 0 || g >= p.num_global) return;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (int64_t)g * p.out_stride + (int64_t)(h * p.G + qi - t * p.G) * D;
  for (int d = threadIdx.x; d < D; d += 32 * kJoinWarps) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) x += so[i][d] * f[i];
    out[d] = __float2bfloat16_rn(x * inv);
  }
}

template <int D, int WQ, int DS, int KG>
cudaError_t launch_cfg(const AttnLaunch& a, cudaStream_t s) {
  using C = Cfg<D, WQ, DS, KG>;
  static std::atomic<uint64_t> done{0};
  const int smem = (int)(C::kRing + C::kMerge + 2 * C::kQ + 1024);
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(split_kernel<D, WQ, DS, KG>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap kmap, vmap;
  if (!encode_pool_maps(a.cache, a.cache.page_size < C::kTN ? a.cache.page_size : C::kTN, &kmap, &vmap))
    return cudaErrorInvalidValue;
  SplitParams P{};
  P.a = a;
  P.info = static_cast<int32_t*>(a.ws);
  P.stats = reinterpret_cast<float*>(P.info + 8 * kSplitCtas);
  P.part = P.stats + (size_t)4 * kSplitCtas * C::kNQ;
  P.wait_ns = kDefaultWaitNs;
  split_kernel<D, WQ, DS, KG><<<kSplitCtas, C::kThreads, smem, s>>>(P, kmap, vmap);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSplitCtas, a.rows.max_q * a.G);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, P, (int)C::kNQ);
}

int query_slots(int64_t queries) { return queries <= 16 ? 16 : queries <= 32 ? 32 : 64; }

}  // namespace

bool attn_split_supported(const AttnLaunch& a, gdn_dtype dtype) {
  const int d = a.cache.d;
  return dtype == GDN_BF16 && (d == 64 || d == 128 || d == 256) && (int64_t)a.rows.max_q * a.G <= 64;
}

size_t attn_split_workspace(const AttnLaunch& a) {
  const size_t q = query_slots((int64_t)a.rows.max_q * a.G);
  return (size_t)kSplitCtas * (8 + 4 * q + 2 * q * a.cache.d) * 4;
}

cudaError_t launch_attn_split(const AttnLaunch& a, cudaStream_t s) {
  // d = 256: two warps share a query group's output columns (16 x 256 accumulators do not fit one)
  switch (a.cache.d + query_slots((int64_t)a.rows.max_q * a.G)) {
    case 64 + 16: return launch_cfg<64, 1, 1, 8>(a, s);
    case 64 + 32: return launch_cfg<64, 2, 1, 4>(a, s);
    case 64 + 64: return launch_cfg<64, 4, 1, 2>(a, s);
    case 128 + 16: return launch_cfg<128, 1, 1, 4>(a, s);
    case 128 + 32: return launch_cfg<128, 2, 1, 4>(a, s);
    case 128 + 64: return launch_cfg<128, 4, 1, 2>(a, s);
    case 256 + 16: return launch_cfg<256, 1, 2, 2>(a, s);
    case 256 + 32: return launch_cfg<256, 2, 2, 2>(a, s);
    case 256 + 64: return launch_cfg<256, 4, 2, 1>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gdn
