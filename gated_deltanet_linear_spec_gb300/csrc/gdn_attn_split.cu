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
// fetched from past the pool and reads as zeros), eight warps compute.  They work transposed,
//   S^T = K Q^T  (tokens x queries),  O^T += V^T P^T  (d x queries),
// so that the tokens fill the m = 16 side of mma.m16n8k16 and 8 queries cost 8 columns, not 16 rows.
// Each warp takes 16 tokens of a tile and up to NQW queries with a running maximum and sum of its
// own; the warps meet only where a unit ends.  The weights enter the second product as a bf16 pair
// (hi + lo), so they keep 16 bits: the product is nearly free here, and one bf16 would cost as much
// accuracy as the output's own rounding.
#include "gdn_tma.cuh"

namespace gdn {

namespace {

constexpr int kSplitCtas = 152;  // one per SM
constexpr uint32_t kSmemBytes = 229600;  // dynamic, behind the alignment: ring and merge buffer
constexpr int kJoinWarps = 8;

template <int D, int NQW, int WQ>
struct Cfg {
  // 8 computing warps; 4 where two tiles at a time would leave the ring too short (d = 256, <= 8 queries)
  static constexpr int kWarps = D == 256 && WQ == 1 ? 4 : 8;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kTN = WQ <= 2 ? 64 : WQ == 4 ? 32 : 16;      // tokens of a tile
  static constexpr int kKT = kTN / 16;                              // 16-token steps of a tile
  static constexpr int kKG = kWarps / WQ;                           // token groups of warps
  static constexpr int kTG = kKG / kKT;                             // tiles worked on at a time
  static constexpr int kNQ = NQW * WQ;                              // queries of a unit, at most
  static constexpr uint32_t kHalf = (uint32_t)kTN * D * 2;          // K (or V) bytes of a stage
  static constexpr int kSlots = kWarps / 2 > WQ ? kWarps / 2 : WQ;  // of the merge buffer, a warp's output each
  static constexpr uint32_t kMerge = (uint32_t)kSlots * NQW * D * 4;
  static constexpr int kFit = (int)((kSmemBytes - kMerge) / (2 * kHalf));
  // A multiple of kTG: a stage is always worked on by the same warps, so none can miss a phase of its barrier.
  static constexpr int kStages = (kFit < 16 ? kFit : 16) / kTG * kTG;
  static constexpr int kNT = NQW / 8;                               // n = 8 tiles of a warp
  static constexpr int kMT = D / 16;
  static_assert(kKT * kTG == kKG && kStages > kTG, "ring too short");
  static constexpr uint32_t kRing = (uint32_t)kStages * 2 * kHalf;
  static_assert(kRing + kMerge <= kSmemBytes, "shared memory");
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
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

// Walks the units of a share: (row, head, tiles [j0, j0 + len) of the unit).
template <int TN>
struct Walk {
  const AttnLaunch& p;
  int64_t left;
  int n, h, j0, len;
  Unit u;
  __device__ Walk(const AttnLaunch& launch, const Share& s) : p(launch), left(s.last - s.first), n(s.row), len(0) {
    if (left <= 0) return;
    u = unit_of<TN>(p, n, nullptr);
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
        u = unit_of<TN>(p, n, nullptr);
      } while (u.tiles == 0);
    }
    len = (int)min((int64_t)u.tiles, left);
  }
  __device__ int tile_at(int j) const { return (j < u.sink_tiles ? j : u.first_tile + j - u.sink_tiles) * TN; }
};

template <int D, int NQW, int WQ>
__global__ void __launch_bounds__(Cfg<D, NQW, WQ>::kThreads, 1)
    split_kernel(SplitParams P, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D, NQW, WQ>;
  constexpr int TN = C::kTN, S = C::kStages, NT = C::kNT, MT = C::kMT;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  float* merge = reinterpret_cast<float*>(ring + C::kRing);
  __shared__ uint64_t full[S], empty[S];
  __shared__ uint32_t held[S];                    // per stage: which of the tile's pages hold tokens
  __shared__ float sm_m[C::kWarps][NQW], sm_l[C::kWarps][NQW];
  __shared__ int dead;
  const AttnLaunch& p = P.a;
  const KvDev& kv = p.cache;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], C::kKT * WQ);
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

  if (warp == C::kWarps) {
    // ---- the fetching warp: lane = (page of the tile, 64-column block, K or V) ----
    constexpr int CB = D / 64;
    const int bi = lane / (2 * CB), cb = (lane >> 1) % CB, is_v = lane & 1;
    const bool active = bi < boxes;
    int it = 0;
    bool ok = true;
    for (Walk<TN> w(p, share); w.valid() && ok; w.next()) {
      const int32_t* row = kv.table + (int64_t)w.u.r.trow * kv.max_pages;
      for (int j = w.j0; j < w.j0 + w.len; ++j, ++it) {
        const int pos = w.tile_at(j) + bi * box;
        int page = 0;
        if (active && pos < w.u.r.kv) page = page_or_null(__ldg(row + pos / ps), kv, p.status);
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
          tc::tma_page(dst, is_v ? &vmap : &kmap, cb * 64, pos % ps, w.h, page > 0 ? page : kv.num_pages, &full[s]);
        }
      }
    }
    // No copy may be in flight when the CTA ends.  Computing warps wait for every stage they use, so
    // this passes at once unless a wait gave up.
    for (int i = max(0, it - S); i < it; ++i) ok &= tc::mbar_wait(&full[i % S], (i / S) & 1, P.wait_ns);
    if (!ok && lane == 0) {
      dead = 1;
      set_status(p.status, GDN_STATUS_WAIT_TIMEOUT);
    }
    return;
  }

  // ---- computing warps ----
  const int wq = warp % WQ, kg = warp / WQ;   // query group, token group
  const int kt = kg % C::kKT, tg = kg / C::kKT;
  const int r8 = lane >> 2, c2 = (lane & 3) * 2;
  const float sl2 = p.scale * 1.4426950408889634f;
  int it = 0;
  bool ok = true;
  for (Walk<TN> w(p, share); w.valid(); w.next()) {
    const KvRow row = w.u.r;
    const int nq = row.len * p.G;
    const int pmin = row.kv - row.len, pmax = row.kv - 1;
    // Q^T as the B operand: query lane / 4, two neighbouring k per register
    uint32_t qf[NT][MT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int qi = wq * NQW + nt * 8 + r8;
      int g = -1;
      if (qi < nq) {
        const int t = qi / p.G;
        g = global_token(RowsDev{nullptr, p.rows.tok}, row.bos + t, p.num_global, p.status);
      }
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)max(g, 0) * p.q_stride +
                               (int64_t)(w.h * p.G + qi % p.G) * D + c2;
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        qf[nt][k][0] = g >= 0 ? __ldg(reinterpret_cast<const uint32_t*>(q + k * 16)) : 0u;
        qf[nt][k][1] = g >= 0 ? __ldg(reinterpret_cast<const uint32_t*>(q + k * 16 + 8)) : 0u;
      }
    }
    float o[NT][MT][4], m[NT][2], l[NT][2];
    int pos_q[NT][2];  // the positions of this thread's query columns
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) pos_q[nt][e] = min(pmin + (wq * NQW + nt * 8 + c2 + e) / p.G, pmax);
    }

    for (int j = w.j0; j < w.j0 + w.len; ++j, ++it) {
      if (C::kTG > 1 && it % C::kTG != tg) continue;
      const int s = it % S;
      ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&full[s], (it / S) & 1, P.wait_ns));
      const int b = w.tile_at(j) + kt * 16;  // first token of this warp's step
      const bool some = ok && b <= pmax && (held[s] >> (kt * 16 / box) & 1u);
      if (some) {
        const uint32_t kbase = tc::smem_addr(ring + (size_t)s * 2 * C::kHalf) + kt * 16 * 128;
        const uint32_t vbase = kbase + C::kHalf;
        // S^T: lanes 0-15 point at rows 0-15 of the left 8 columns, lanes 16-31 of the right 8
        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
        {
          const int r = lane & 15;
          const uint32_t base = kbase + r * 128;
#pragma unroll
          for (int k = 0; k < MT; ++k) {
            uint32_t a[4];
            ldsm4(a, base + (k >> 2) * TN * 128 + ((((k & 3) * 2 + (lane >> 4)) ^ (r & 7)) << 4));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(sc[nt], a, qf[nt][k][0], qf[nt][k][1]);
          }
        }
        // which of the step's tokens a query sees; `part`: not every query sees every token
        const bool part = b + 15 > pmin || (p.window > 0 && b <= pmax - p.window && b + 15 >= p.sinks);
        uint32_t vmask0 = 0xffffffffu, vmask1 = 0xffffffffu;
        bool vis[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = sc[nt][e] * sl2;
            vis[nt][e] = true;
            if (part) {
              const int tok = b + r8 + (e >> 1) * 8, at = pos_q[nt][e & 1];
              vis[nt][e] = tok <= at && (p.window <= 0 || tok > at - p.window || tok < p.sinks);
              if (!vis[nt][e]) x = -INFINITY;
            }
            sc[nt][e] = x;
          }
        }
        float mx[NT][2];
        bool grew = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(sc[nt][e], sc[nt][e + 2]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            mx[nt][e] = fmaxf(m[nt][e], x);
            grew |= mx[nt][e] > m[nt][e];
          }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              a[e] = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - mx[nt][e]);
              m[nt][e] = mx[nt][e];
              l[nt][e] *= a[e];
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[nt][i][0] *= a[0];
              o[nt][i][1] *= a[1];
              o[nt][i][2] *= a[0];
              o[nt][i][3] *= a[1];
            }
          }
        }
        // P^T as the B operand: transposed 8 x 8 blocks of the score fragments, as hi + lo
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float mm = m[nt][e & 1];
            e4[e] = ex2(sc[nt][e] - (mm == -INFINITY ? 0.f : mm));
          }
          l[nt][0] += e4[0] + e4[2];
          l[nt][1] += e4[1] + e4[3];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t hi = pack2(e4[2 * hf], e4[2 * hf + 1]);
            const uint32_t lo = pack2(e4[2 * hf] - bf_lo(hi), e4[2 * hf + 1] - bf_hi(hi));
            ph[nt][hf] = transpose8(hi);
            pl[nt][hf] = transpose8(lo);
          }
        }
        if (part) {
          // tokens past the row's end hold anything: their values do not enter the products
          const int tok = b + c2;
          vmask0 = (tok <= pmax ? 0xffffu : 0u) | (tok + 1 <= pmax ? 0xffff0000u : 0u);
          vmask1 = (tok + 8 <= pmax ? 0xffffu : 0u) | (tok + 9 <= pmax ? 0xffff0000u : 0u);
        }
        // O^T += V^T P^T: lanes 0-7, 8-15, 16-23, 24-31 point at (tokens 0-7, left 8 columns),
        // (0-7, right), (8-15, left), (8-15, right); the transposing load makes d the row
        const int r = (lane & 7) + ((lane >> 4) << 3);
        const uint32_t base = vbase + r * 128;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          uint32_t a[4];
          ldsm4t(a, base + (i >> 2) * TN * 128 + ((((i & 3) * 2 + ((lane >> 3) & 1)) ^ (r & 7)) << 4));
          if (part) {
            a[0] &= vmask0;
            a[1] &= vmask0;
            a[2] &= vmask1;
            a[3] &= vmask1;
            const bool odd = not_finite2(a[0]) || not_finite2(a[1]) || not_finite2(a[2]) || not_finite2(a[3]);
            if (__any_sync(0xffffffffu, odd)) {
              // An infinity or NaN that some query of the step must not see (0 times it is NaN): one
              // token at a time, added only where it is seen.
#pragma unroll 1
              for (int t = 0; t < 16; ++t) {
                const uint32_t half = (t & 1) ? 0xffff0000u : 0xffffu;
                const uint32_t keep = ((t & 7) >> 1) == (lane & 3) ? half : 0u;
                uint32_t one[4];
                one[0] = t < 8 ? a[0] & keep : 0u;
                one[1] = t < 8 ? a[1] & keep : 0u;
                one[2] = t < 8 ? 0u : a[2] & keep;
                one[3] = t < 8 ? 0u : a[3] & keep;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float x[4] = {0.f, 0.f, 0.f, 0.f};
                  mma16816(x, one, ph[nt][0], ph[nt][1]);
                  mma16816(x, one, pl[nt][0], pl[nt][1]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const int at = pos_q[nt][e & 1], tk = b + t;
                    if (tk <= at && (p.window <= 0 || tk > at - p.window || tk < p.sinks)) o[nt][i][e] += x[e];
                  }
                }
              }
              continue;
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(o[nt][i], a, ph[nt][0], ph[nt][1]);
            mma16816(o[nt][i], a, pl[nt][0], pl[nt][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty[s]);
    }

    // ---- the unit's piece ends: join the warps of a query group, token groups pairwise ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
      }
    if (!ok && lane == 0) {
      dead = 1;
      set_status(p.status, GDN_STATUS_WAIT_TIMEOUT);
    }
#pragma unroll
    for (int step = C::kKG / 2; step >= 1; step >>= 1) {
      compute_bar<C::kWarps>();
      if (kg >= step && kg < 2 * step) {
        const int slot = (kg - step) * WQ + wq;
        float4* b4 = reinterpret_cast<float4*>(merge) + (size_t)slot * NT * MT * 32 + lane;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < MT; ++i)
            b4[(nt * MT + i) * 32] = make_float4(o[nt][i][0], o[nt][i][1], o[nt][i][2], o[nt][i][3]);
        if (lane < 4)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              sm_m[slot][nt * 8 + c2 + e] = m[nt][e];
              sm_l[slot][nt * 8 + c2 + e] = l[nt][e];
            }
      }
      compute_bar<C::kWarps>();
      if (kg < step) {
        const int slot = kg * WQ + wq;
        const float4* b4 = reinterpret_cast<const float4*>(merge) + (size_t)slot * NT * MT * 32 + lane;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float a[2], c[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float m2 = sm_m[slot][nt * 8 + c2 + e], mn = fmaxf(m[nt][e], m2);
            a[e] = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - mn);
            c[e] = m2 == -INFINITY ? 0.f : ex2(m2 - mn);
            l[nt][e] = l[nt][e] * a[e] + sm_l[slot][nt * 8 + c2 + e] * c[e];
            m[nt][e] = mn;
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const float4 v = b4[(nt * MT + i) * 32];
            o[nt][i][0] = o[nt][i][0] * a[0] + v.x * c[0];
            o[nt][i][1] = o[nt][i][1] * a[1] + v.y * c[1];
            o[nt][i][2] = o[nt][i][2] * a[0] + v.z * c[0];
            o[nt][i][3] = o[nt][i][3] * a[1] + v.w * c[1];
          }
        }
      }
    }
    compute_bar<C::kWarps>();
    if (kg == 0 && !*(volatile int*)&dead) {
      const bool whole = w.j0 == 0 && w.len == w.u.tiles;
      // rows of queries in shared memory, then 16-byte stores
      float* mine = merge + (size_t)wq * NQW * D;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) f[e] = !whole ? 1.f : l[nt][e] == 0.f ? 0.f : 1.f / l[nt][e];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mine[(nt * 8 + c2 + (e & 1)) * D + i * 16 + r8 + (e >> 1) * 8] = o[nt][i][e] * f[e & 1];
      }
      __syncwarp();
      if (whole) {
#pragma unroll 1
        for (int v = lane; v < NQW * D / 8; v += 32) {
          const int q = v / (D / 8), d0 = (v % (D / 8)) * 8, qi = wq * NQW + q;
          if (qi >= nq) continue;
          const int t = qi / p.G;
          const int g = p.rows.tok ? __ldg(p.rows.tok + row.bos + t) : row.bos + t;
          if (g < 0 || g >= p.num_global) continue;
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + (int64_t)g * p.out_stride +
                                    (int64_t)(w.h * p.G + qi - t * p.G) * D + d0) = tc::pack8(mine + q * D + d0);
        }
      } else {
        const int slot = 2 * blockIdx.x + (w.j0 == 0 ? 1 : 0);
        float4* dst = reinterpret_cast<float4*>(P.part + ((size_t)slot * C::kNQ + wq * NQW) * D);
#pragma unroll 1
        for (int v = lane; v < NQW * D / 4; v += 32) dst[v] = reinterpret_cast<const float4*>(mine)[v];
        if (lane < 4)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float* st = P.stats + ((size_t)slot * C::kNQ + wq * NQW + nt * 8 + c2 + e) * 2;
              st[0] = m[nt][e];
              st[1] = l[nt][e];
            }
        if (w.j0 == 0 && wq == 0 && lane == 0) {
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
    const float a = m == -INFINITY ? 0.f : ex2(m - mn), b = m2 == -INFINITY ? 0.f : ex2(m2 - mn);
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
    f[i] = sm[i] == -INFINITY ? 0.f : ex2(sm[i] - M);
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

template <int D, int NQW, int WQ>
cudaError_t launch_cfg(const AttnLaunch& a, cudaStream_t s) {
  using C = Cfg<D, NQW, WQ>;
  static std::atomic<uint64_t> done{0};
  const int smem = (int)(C::kRing + C::kMerge + 1024);
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(split_kernel<D, NQW, WQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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
  split_kernel<D, NQW, WQ><<<kSplitCtas, C::kThreads, smem, s>>>(P, kmap, vmap);
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

int query_slots(int64_t queries) { return queries <= 8 ? 8 : queries <= 16 ? 16 : queries <= 32 ? 32 : 64; }

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
  const int q = query_slots((int64_t)a.rows.max_q * a.G);
  // 16 queries per warp where their accumulators fit the registers (d <= 128), else 8
  switch (a.cache.d * 128 + q) {
    case 64 * 128 + 8: return launch_cfg<64, 8, 1>(a, s);
    case 64 * 128 + 16: return launch_cfg<64, 16, 1>(a, s);
    case 64 * 128 + 32: return launch_cfg<64, 16, 2>(a, s);
    case 64 * 128 + 64: return launch_cfg<64, 16, 4>(a, s);
    case 128 * 128 + 8: return launch_cfg<128, 8, 1>(a, s);
    case 128 * 128 + 16: return launch_cfg<128, 16, 1>(a, s);
    case 128 * 128 + 32: return launch_cfg<128, 16, 2>(a, s);
    case 128 * 128 + 64: return launch_cfg<128, 16, 4>(a, s);
    case 256 * 128 + 8: return launch_cfg<256, 8, 1>(a, s);
    case 256 * 128 + 16: return launch_cfg<256, 8, 2>(a, s);
    case 256 * 128 + 32: return launch_cfg<256, 8, 4>(a, s);
    case 256 * 128 + 64: return launch_cfg<256, 8, 8>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gdn
