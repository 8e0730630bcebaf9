// gdn_attn_split.cu -- attention of decode and verify rows over the paged cache (bf16, d = 64, 128, 256).
//
// Up to 64 queries (new tokens x q-heads of one kv-head) share every key and value, so the bytes of
// the cache bound the kernel: 4 flops per query per element against 2 bytes, far under the tensor
// cores' ratio.  What matters is that every SM streams its share of the cache without a pause.
//
// Work.  A unit is one (row, kv-head): the 32-token tiles that its queries see, window and first
// tokens included.  All units' tiles laid end to end are dealt out evenly, so ragged lengths and a
// single long row load the SMs alike.  A share's piece of a unit that is not the whole unit leaves
// (m, l, o) in the workspace; the join kernel adds a unit's pieces in the order of the workers, so
// results do not depend on timing.
//
// A CTA (one per SM) holds 1 to 6 workers, each with a share of its own: one warp fetches pages by TMA
// into a short ring of stages (a NULL page is fetched from past the pool and reads as zeros) and the
// queries of the next unit; one warp per 16 queries computes, 32 tokens a step, with mma.m16n8k16 and a
// running maximum and sum of its own.  No warp waits for another, and an SM's workers cover one another's starts
// and ends of units (with 8 warps sharing a tile and meeting at every unit's end, 64 decode rows took 96 us).
// They are one CTA so that their computing warps spread evenly over the SM's four schedulers.  The weights enter
// the second product as a bf16 pair (hi + lo), so they keep 16 bits: the product is nearly free here, and one
// bf16 would cost as much accuracy as the output's own rounding.
// Measured with the join (L2 flushed before each call): 64 decode rows over 512 to 8192 tokens (32 q-heads, 4
// kv-heads, d = 128, pages of 16) 68 us = 5.5 TB/s; 64 rows of 4 verify tokens over 1000 to 16384 131 us = 5.7; four
// rows over 65536 to 131072 tokens (d = 256) 136 us = 6.4; 128 windowed rows (d = 64) 53 us = 4.5.  Between its
// start (about 3 us until every worker knows its share and has a page) and its last workers the kernel
// streams at 6.2 to 6.9 TB/s, what a copy reaches; more workers or one product instead of the pair change nothing.
#include <algorithm>

#include "gdn_attn_share.cuh"
#include "gdn_tma.cuh"

namespace gdn {

namespace {

using namespace split;

// NW workers of WQ groups of 16 queries x DS slices of the values' columns, a computing warp each.
template <int D, int WQ, int DS, int NW>
struct Cfg {
  static constexpr int kTeam = WQ * DS;                             // computing warps of a worker
  static constexpr int kThreads = 32 * NW * (kTeam + 1);
  static constexpr int kWorkers = NW;
  static constexpr int kNQ = 16 * WQ;                               // queries of a unit, at most
  static constexpr int kDV = D / DS;                                // value columns of a warp
  static constexpr uint32_t kHalf = (uint32_t)kTN * D * 2;          // K (or V) bytes of a stage
  static constexpr uint32_t kPitch = D * 2 + 16;                    // bytes of a query: rows 16 bytes apart mod 128
  static constexpr uint32_t kQ = kNQ * kPitch;
  // what a CTA with rings of s stages takes (struct Small's sizes among it)
  static constexpr uint32_t bytes(int s) { return NW * (s * 2 * kHalf + kQ + (17 * s + 16 + 4 * kNQ + 7) / 8 * 8 + 48) + 16; }
  static constexpr int most() {
    int s = 8;
    while (bytes(s) > 232448) --s;
    return s;
  }
  static constexpr int kStages = most();
  static constexpr uint32_t kRing = (uint32_t)kStages * 2 * kHalf;  // of a worker
  static_assert(kStages >= 2, "ring too short");
};

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
  asm(
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
// One 32-token step's second product, O += P V.  PART: some query does not see some token, so the
// values must not reach it whatever they hold.
template <bool PART, int DV, int CB>
__device__ __forceinline__ void values_step(float (&o)[DV / 8][4], const uint32_t (&ph)[2][4], const uint32_t (&pl)[2][4],
                                            uint32_t vbase, int col0, int b, const int (&pos)[2], int pmax, int window,
                                            int sinks) {
  const int lane = threadIdx.x & 31, c2 = (lane & 3) * 2;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    // lanes 0-7, 8-15, 16-23, 24-31 point at (tokens 0-7, left 8 columns), (8-15, left), (0-7, right),
    // (8-15, right); the transposing load puts two tokens of a column into a register
    const int r = (lane & 7) + (((lane >> 3) & 1) << 3);
    const uint32_t base = vbase + (half * 2 + (r >> 3)) * CB * 1024 + (r & 7) * 128;
    const int t0 = b + half * 16;
    uint32_t m0 = 0xffffffffu, m1 = 0xffffffffu;
    if (PART) {  // tokens past the row's end hold anything
      m0 = (t0 + c2 <= pmax ? 0xffffu : 0u) | (t0 + c2 + 1 <= pmax ? 0xffff0000u : 0u);
      m1 = (t0 + c2 + 8 <= pmax ? 0xffffu : 0u) | (t0 + c2 + 9 <= pmax ? 0xffff0000u : 0u);
    }
    // Two 16-column blocks at a time: the four accumulators take their hi products, then their lo
    // ones, so no product waits for the one just before it.
#pragma unroll
    for (int i = 0; i < DV / 16; i += 2) {
      uint32_t v[2][4];
      bool odd = false;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int chunk = col0 / 8 + (i + u) * 2 + (lane >> 4);
        ldsm4t(v[u], base + (chunk >> 3) * 1024 + (((chunk & 7) ^ (r & 7)) << 4));
        if (PART) {
          v[u][0] &= m0;
          v[u][1] &= m1;
          v[u][2] &= m0;
          v[u][3] &= m1;
          odd |= not_finite2(v[u][0]) || not_finite2(v[u][1]) || not_finite2(v[u][2]) || not_finite2(v[u][3]);
        }
      }
      if (PART && __any_sync(0xffffffffu, odd)) {
        // An infinity or NaN that some query of the step must not see (0 times it is NaN): one token
        // at a time, added only where it is seen.
#pragma unroll 1
        for (int t = 0; t < 16; ++t) {
          const uint32_t keep = ((t & 7) >> 1) == (lane & 3) ? ((t & 1) ? 0xffff0000u : 0xffffu) : 0u;
          const uint32_t lo = t < 8 ? keep : 0u, hi = t < 8 ? 0u : keep;
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816(x, ph[half], v[n >> 1][2 * (n & 1)] & lo, v[n >> 1][2 * (n & 1) + 1] & hi);
            mma16816(x, pl[half], v[n >> 1][2 * (n & 1)] & lo, v[n >> 1][2 * (n & 1) + 1] & hi);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = pos[e >> 1], tk = t0 + t;
              if (tk <= at && (window <= 0 || tk > at - window || tk < sinks)) o[2 * i + n][e] += x[e];
            }
          }
        }
        continue;
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) mma16816(o[2 * i + n], ph[half], v[n >> 1][2 * (n & 1)], v[n >> 1][2 * (n & 1) + 1]);
#pragma unroll
      for (int n = 0; n < 4; ++n) mma16816(o[2 * i + n], pl[half], v[n >> 1][2 * (n & 1)], v[n >> 1][2 * (n & 1) + 1]);
    }
  }
}

// What a CTA keeps in shared memory behind its rings and queries.
template <typename C>
struct Small {
  struct Worker {
    uint64_t full[C::kStages], empty[C::kStages], qfull, qempty;
    int qtok[C::kNQ];          // the queries' global tokens, -1 for none
    uint8_t held[C::kStages];  // per stage: which halves of the tile lie in pages that hold tokens
  } worker[C::kWorkers];
  Deal deal;
  Share<false> shares[C::kWorkers];
};

template <int D, int WQ, int DS, int NW>
__global__ void __launch_bounds__(Cfg<D, WQ, DS, NW>::kThreads, 1)
    split_kernel(SplitParams P, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D, WQ, DS, NW>;
  constexpr int S = C::kStages, DV = C::kDV;
  extern __shared__ __align__(1024) uint8_t smem[];
  Small<C>& small = *reinterpret_cast<Small<C>*>(smem + NW * (C::kRing + C::kQ));
  const AttnLaunch& p = P.a;
  const KvDev& kv = p.cache;
  // The warp's number comes from a shuffle, so that the compiler takes it as one value of the warp.  (In an early form
  // that took it as threadIdx.x / 32, nvcc 13.0 got the range of an index into shared memory wrong under nested
  // conditions, and the index left its array.)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid < NW) {
    for (int i = 0; i < S; ++i) {
      tc::mbar_init(&small.worker[tid].full[i], 1);
      tc::mbar_init(&small.worker[tid].empty[i], C::kTeam);
    }
    tc::mbar_init(&small.worker[tid].qfull, 1);
    tc::mbar_init(&small.worker[tid].qempty, C::kTeam);
    tc::mbar_init_fence();
  }
  if (tid == 32) {
    tc::prefetch_map(&kmap);
    tc::prefetch_map(&vmap);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what lies before this overlaps the kernel before this one
  if (tid < NW) P.info[(blockIdx.x * NW + tid) * 8] = 0;
  // (the sums of find_shares lie where the first worker's ring will be)
  find_shares<0, NW, C::kThreads>(p, reinterpret_cast<int64_t*>(smem), small.deal, small.shares);
  const bool fetches = warp >= NW * C::kTeam;
  const int wk = fetches ? warp - NW * C::kTeam : warp / C::kTeam;  // the warp's worker
  auto& sm = small.worker[wk];
  const Share<false>& share = small.shares[wk];
  uint8_t* ring = smem + wk * C::kRing;
  uint8_t* qbuf = smem + NW * C::kRing + wk * C::kQ;
  const int ps = kv.page_size;
  const int box = min(ps, kTN);      // tokens of one copy
  const int boxes = kTN / box;       // pages of a tile
  const int shift = __ffs(ps) - 1;

  if (fetches) {
    // ---- the fetching warp: lane = (page of the tile, K or V) ----
    const int bi = lane >> 1, is_v = lane & 1, spp = slabs_per_page(kv);
    const int none = (kv.num_pages - 1) * spp + kv.Hkv;  // a slab past the pool
    const bool active = bi < boxes;
    int it = 0, seg = 0;
    bool ok = true;
    for (Walk<0> w(p, share); w.valid() && ok; w.next(), ++seg) {
      // 32 table entries are held, one per lane, and the 32 behind them are on their way
      const int32_t* row = kv.table + (int64_t)w.u.r.trow * kv.max_pages;
      const int entries = (w.u.r.kv + ps - 1) >> shift;
      int eb = w.tile_at(w.j0) >> shift;
      int ids = eb + lane < entries ? load(row + eb + lane) : 0;
      int ahead = eb + 32 + lane < entries ? load(row + eb + 32 + lane) : 0;
      // the unit's queries
      const int nq = w.u.r.len * p.G;
      int g[2];
      int rows = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int qi = lane + 32 * u;
        g[u] = -1;
        if (qi < nq) g[u] = kv_token(p.rows, w.u.r.bos + qi / p.G, p.num_global, p.status);
        rows += __popc(__ballot_sync(0xffffffffu, g[u] >= 0));
      }
      ok = seg == 0 || tc::mbar_wait(&sm.qempty, (seg - 1) & 1, P.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (lane + 32 * u < C::kNQ) sm.qtok[lane + 32 * u] = g[u];
      __syncwarp();
      if (lane == 0) tc::expect_tx(&sm.qfull, (uint32_t)rows * D * 2);
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int qi = lane + 32 * u;
        if (g[u] >= 0)
          tc::bulk_g2s(qbuf + qi * C::kPitch,
                       static_cast<const __nv_bfloat16*>(p.q) + (int64_t)g[u] * p.q_stride +
                           (int64_t)(w.h * p.G + qi % p.G) * D,
                       D * 2, &sm.qfull);
      }
      for (int j = w.j0; j < w.j0 + w.len; ++j, ++it) {
        const int pos = w.tile_at(j) + bi * box;
        const int e = w.tile_at(j) >> shift;
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
        page = active && pos < w.u.r.kv ? page_or_null(page, kv, p.status) : 0;
        const int s = it % S;
        ok = it < S || tc::mbar_wait(&sm.empty[s], ((it / S) - 1) & 1, P.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t have = __ballot_sync(0xffffffffu, page > 0);
        const uint32_t mask = (have & 1u) | (have >> 1 & 2u);  // (lanes 0 and 2: the tile's one or two pages)
        if (lane == 0) {
          sm.held[s] = (uint8_t)mask;
          tc::expect_tx(&sm.full[s], 2 * C::kHalf);
        }
        __syncwarp();
        if (active) {
          uint8_t* dst = ring + (size_t)s * 2 * C::kHalf + is_v * C::kHalf + (size_t)bi * box * D * 2;
          tc::tma_page(dst, is_v ? &vmap : &kmap, pos & (ps - 1), page > 0 ? page * spp + w.h : none, &sm.full[s]);
        }
      }
    }
    // No copy may be in flight when the CTA ends.  Computing warps wait for every stage they use, so
    // this passes at once unless a wait gave up.
    for (int i = max(0, it - S); i < it; ++i) ok &= tc::mbar_wait(&sm.full[i % S], (i / S) & 1, P.wait_ns);
    if (seg > 0) ok &= tc::mbar_wait(&sm.qfull, (seg - 1) & 1, P.wait_ns);
    if (!ok) set_status(p.status, GDN_STATUS_WAIT_TIMEOUT);
    return;
  }

  // ---- computing warps ----
  const int ds = warp % DS, wq = (warp - wk * C::kTeam) / DS;
  const int r8 = lane >> 2, c2 = (lane & 3) * 2;
  const int bshift = __ffs(box) - 1;
  const float sl2 = p.scale * 1.4426950408889634f;
  int it = 0, seg = 0;
  bool ok = true;
  for (Walk<0> w(p, share); w.valid(); w.next(), ++seg) {
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
    ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&sm.qfull, seg & 1, P.wait_ns));
    const uint32_t qbase =
        tc::smem_addr(qbuf) + (wq * 16 + (lane & 15)) * C::kPitch + (lane >> 4) * 16;

    for (int j = w.j0; j < w.j0 + w.len; ++j, ++it) {
      const int s = it % S;
      ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&sm.full[s], (it / S) & 1, P.wait_ns));
      const int b = w.tile_at(j);
      // a page is 16 tokens or more: the step's two halves may differ in whether theirs is NULL
      const uint32_t hm = sm.held[s];
      const bool have0 = hm & 1u, have1 = hm >> (16 >> bshift) & 1u;
      if (ok && (have0 || have1)) {
        const uint32_t kbase = tc::smem_addr(ring + (size_t)s * 2 * C::kHalf);
        const uint32_t vbase = kbase + C::kHalf;
        // S = Q K^T.  K as the B operand: lanes 0-7, 8-15, 16-23, 24-31 point at (tokens 0-7, left 8
        // columns), (0-7, right), (8-15, left), (8-15, right) of 16 tokens.
        float sc[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
        {
          const int r = (lane & 7) + ((lane >> 4) << 3);
          const uint32_t base = kbase + (r >> 3) * (D / 64) * 1024 + (r & 7) * 128;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t a[4], k0[4], k1[4];
            const uint32_t at =
                base + (k >> 2) * 1024 + ((((k & 3) * 2 + ((lane >> 3) & 1)) ^ (r & 7)) << 4);
            ldsm4(a, qbase + k * 32);
            ldsm4(k0, at);
            ldsm4(k1, at + 2 * (D / 64) * 1024);
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
          values_step<true, DV, D / 64>(o, ph, pl, vbase, ds * DV, b, pos, pmax, p.window, p.sinks);
        else
          values_step<false, DV, D / 64>(o, ph, pl, vbase, ds * DV, b, pos, pmax, p.window, p.sinks);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.empty[s]);
    }
    // ---- the unit's piece ends ----
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }
    if (!ok) {
      set_status(p.status, GDN_STATUS_WAIT_TIMEOUT);
    } else {
      const bool whole = w.j0 == 0 && w.len == w.u.tiles;
      const int slot = 2 * (blockIdx.x * NW + wk) + (w.j0 == 0 ? 1 : 0);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int qi = wq * 16 + r8 + 8 * e;
        const int g = sm.qtok[qi];
        if (whole && g >= 0) {
          const float f = l[e] == 0.f ? 0.f : 1.f / l[e];
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (int64_t)g * p.out_stride +
                               (int64_t)(w.h * p.G + qi % p.G) * D + ds * DV + c2;
#pragma unroll
          for (int i = 0; i < DV / 8; ++i)
            *reinterpret_cast<uint32_t*>(out + i * 8) = pack2(o[i][2 * e] * f, o[i][2 * e + 1] * f);
        } else if (!whole && qi < nq) {
          float* part = P.part + ((size_t)slot * C::kNQ + qi) * D + ds * DV + c2;
#pragma unroll
          for (int i = 0; i < DV / 8; ++i)
            *reinterpret_cast<float2*>(part + i * 8) = make_float2(o[i][2 * e], o[i][2 * e + 1]);
          if (ds == 0 && c2 == 0)
            *reinterpret_cast<float2*>(P.stats + ((size_t)slot * C::kNQ + qi) * 2) = make_float2(m[e], l[e]);
        }
      }
      if (!whole && w.j0 == 0 && wq == 0 && ds == 0 && lane == 0) {
        int32_t* info = P.info + (blockIdx.x * NW + wk) * 8;
        info[1] = row.bos;
        info[2] = nq;
        info[3] = w.h;
        info[5] = 0;
        info[4] = small.deal.owner(w.unit_last(share));  // the worker with the unit's last tile
        info[0] = 1;
      }
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sm.qempty);
  }
}

// Queries of a unit, at most (with max_q = 0 every row is a bad one, and reported).
int64_t queries_of(const AttnLaunch& a) {
  return a.few > 0 ? a.few : std::max<int64_t>(1, (int64_t)a.rows.max_q * a.G);
}

template <int D, int WQ, int DS, int NW>
cudaError_t launch_cfg(const AttnLaunch& a, cudaStream_t s) {
  using C = Cfg<D, WQ, DS, NW>;
  static std::atomic<uint64_t> done{0};
  constexpr int smem = (int)(NW * (C::kRing + C::kQ) + sizeof(Small<C>));
  static_assert(smem <= 232448 && C::kThreads / 32 * 8 <= (int)C::kRing, "shared memory");
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(split_kernel<D, WQ, DS, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap kmap, vmap;
  if (!encode_pool_maps(a.cache, a.cache.page_size < kTN ? a.cache.page_size : kTN, &kmap, &vmap))
    return cudaErrorInvalidValue;
  SplitParams P{};
  P.a = a;
  P.info = static_cast<int32_t*>(a.ws);
  P.stats = reinterpret_cast<float*>(P.info + 8 * kSms * NW);
  P.part = P.stats + (size_t)4 * kSms * NW * C::kNQ;
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
  if ((e = cudaLaunchKernelEx(&cfg, split_kernel<D, WQ, DS, NW>, P, kmap, vmap)) != cudaSuccess) return e;
  cfg.gridDim = dim3(kSms * NW, join_rows(kSms * NW, (int)queries_of(a)));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<__nv_bfloat16, D / 32, D>, P, (int)C::kNQ);
}

int query_slots(int64_t queries) { return queries <= 16 ? 16 : queries <= 32 ? 32 : 64; }

}  // namespace

// A call of long rows may hold one-token rows too (a GDN batch's decode rows come with its prompts).  As prompts they
// take a CTA per row and kv-head, 128 or 256 queries wide.  The host knows the rows' count, their tokens and the longest:
// from 5 rows on that have less than half the longest's tokens on average, some are short and the call is split.  Decode
// rows over 512 to 8192 tokens (32 q-heads, 4 kv-heads, d = 128), all as prompts and split: beside a 1024-token prompt 2
// rows 76 and 55 us, 4 101 and 59, 16 140 and 73, 64 164 and 123; beside one of 4096 2 rows 158 and 178, 4 185 and 182,
// 16 212 and 195; 300 new tokens at 2000 2 rows 48 and 59, 4 70 and 63, 16 125 and 78.  Where no row is short the two more
// launches lose 9 to 11 us (3 ragged prompts: 48 and 57; 12 of 100 to 1200 tokens, which this rule does not split: 113 and
// 125).
int32_t attn_few(const AttnLaunch& a, gdn_dtype dtype) {
  const bool short_ones = 2 * (int64_t)a.rows.num_tokens < (int64_t)a.rows.num_seqs * a.rows.max_q;
  if (!attn_prompt_supported(a, dtype) || attn_split_supported(a, dtype) || a.G > 64 || a.rows.num_seqs < 5 || !short_ones)
    return 0;
  return query_slots(a.G);
}

bool attn_split_supported(const AttnLaunch& a, gdn_dtype dtype) {
  const int d = a.cache.d;
  return dtype == GDN_BF16 && (d == 64 || d == 128 || d == 256) && (int64_t)a.rows.max_q * a.G <= 64;
}

namespace {

// d = 256: two warps share a query group's output columns (16 x 256 accumulators do not fit one).
// Workers: as many as leave each a ring of 3 stages or more and the registers (168 a thread).
template <typename F>
auto pick(int d, int slots, F f) {
  if (d == 64) return slots == 16 ? f(Cfg<64, 1, 1, 6>{}) : slots == 32 ? f(Cfg<64, 2, 1, 4>{}) : f(Cfg<64, 4, 1, 2>{});
  if (d == 128) return slots == 16 ? f(Cfg<128, 1, 1, 4>{}) : slots == 32 ? f(Cfg<128, 2, 1, 4>{}) : f(Cfg<128, 4, 1, 2>{});
  return slots == 16 ? f(Cfg<256, 1, 2, 2>{}) : slots == 32 ? f(Cfg<256, 2, 2, 2>{}) : f(Cfg<256, 4, 2, 1>{});
}

template <int D, int WQ, int DS, int NW>
cudaError_t launch_picked(Cfg<D, WQ, DS, NW>, const AttnLaunch& a, cudaStream_t s) {
  return launch_cfg<D, WQ, DS, NW>(a, s);
}

}  // namespace

size_t attn_split_workspace(const AttnLaunch& a) {
  const int q = query_slots(queries_of(a));
  const size_t workers = (size_t)kSms * pick(a.cache.d, q, [](auto c) { return decltype(c)::kWorkers; });
  return workers * (8 + 4 * (size_t)q + 2 * (size_t)q * a.cache.d) * 4;
}

cudaError_t launch_attn_split(const AttnLaunch& a, cudaStream_t s) {
  return pick(a.cache.d, query_slots(queries_of(a)), [&](auto c) { return launch_picked(c, a, s); });
}

}  // namespace gdn
