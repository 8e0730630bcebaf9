// gdn_attn_shared.cu -- groups' queries over what their rows share, and rows' over their own tokens, on tcgen05 (bf16, d = 64,
// 128, 256).
//
// The queries of a group's rows stand one after the other, 256 (d = 256: 128) to a CTA, and every shared key and value is read
// once for all of them: 4 d flops per score, so the tensor core bounds it as it does prompts, and tiles, products and
// softmax are those of gdn_attn_prompt.cu.  A query stands behind all shared tokens, so only a window hides some of them; a
// row's own tokens are causal.
//
// Units (part, kv-head, 256 queries) are dealt out as in gdn_attn_share.cuh, 64-token tiles laid end to end, so that all SMs
// end together whatever the groups' sizes are; a unit's pieces meet in the join of parts.  A tile of 128 queries that a unit
// does not have (few queries, a row's own part) takes no part in its steps; a step takes little less time for that, as
// its scores, softmax and second product wait for one another.
//
// Weights go into the second product as two bf16 terms, 16 bits, in calls whose rows attention without groups gives as many:
// the scores' 64 columns of TMEM hold both.  With one term the first call below took 145 us and the second 35.
//
// Measured (32 q-heads, 4 kv-heads, d = 128): 64 rows of 4 tokens behind 32768 shared ones 164 us, 0.84 PFLOP/s; 64 of 1 behind
// 8200, up to 1024 own tokens each, 39 us (two thirds of the tiles are own ones).  With 128 tokens a step, which leave room for
// one score buffer, the first took 155 us (151 at that time, with one term); with the rows' own parts on mma.sync beside
// this kernel's end 158 and the second 49 (151 and 40).
#include <algorithm>
#include <atomic>

#include "gdn_attn_share.cuh"
#include "gdn_attn_tile.cuh"
#include "gdn_testing.h"

namespace gdn {

namespace {

using namespace tile;

// Beginning a unit -- its queries, the first scores, its results -- takes about as long as so many 64-token steps: steps of two
// query tiles, where the call has units of two, or the shorter ones of one.  (16 groups of 4 rows of 4 tokens behind 8192, 20 own
// ones each: 77 us with 4, 83 with 2; behind 512 31.5 and 28.2.  One group of 64 rows of 1 behind 8200: 42.3 with 4, 39.1 with 2.)
constexpr int kBegin = 2, kBeginOne = 4;

// K and V pairs in the ring: 128 KB, which keeps HBM busy under short steps too.
__host__ __device__ constexpr int phases_of(int d) { return 512 / d; }

struct SharedParams {
  AttnLaunch a;
  float* o;      // [2 * kSms][D / 4][kRows][4]
  float* stats;  // [2 * kSms][kRows][2]
  uint64_t wait_ns;
  int32_t stop_tile;  // fetches end in front of a CTA's so manieth tile; -1: they do not
};
// Test hook (gdn_testing.h).
std::atomic<uint64_t> g_test_wait_ns{0};
std::atomic<int32_t> g_test_stop_tile{-1};

template <int D>
struct Small {
  uint64_t full[2 * phases_of(D)], empty[2 * phases_of(D)];
  uint64_t checked[phases_of(D)];  // of a V tile
  uint64_t q_ready[2], drain[2];
  uint64_t s_ready[2][2], p_ready[2][2], pv_done[2][2];  // [query tile][score buffer]
  int64_t sum[Cfg<D>::kThreads / 32];
  split::Deal deal;
  split::Share<true> share;
  uint32_t bad[phases_of(D)][2];  // listed tokens of a V tile
  uint32_t held[16];              // per tile, counted over all units, % 16: which of its pages hold tokens
  uint32_t tmem;
};

// PAIR: weights go into the second product as two bf16 terms (over the scores, which take twice the room).
template <int D, bool PAIR>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    shared_kernel(SharedParams P, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D>;
  using Units = split::Walk<C::kRows, true, kTN>;
  constexpr int NT = C::kTiles, kPh = phases_of(D), R = 2 * kPh, CB = D / 64;
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
  const PartRec* near = p.part.plan_here ? plan_here<C::kThreads>(p, reinterpret_cast<int*>(ring)) : nullptr;
  split::find_shares<C::kRows, 1, C::kThreads, true, kTN, kBegin, NT == 2 ? kBeginOne : kBegin>(p, sm.sum, sm.deal, &sm.share, near);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sm.tmem;
  const int ps = kv.page_size, shift = __ffs(ps) - 1, box = min(ps, kTN), boxes = kTN / box;
  const int bshift = __ffs(box) - 1;

  Units w(p, sm.share, sm.deal.start);
  bool ok = true;
  uint32_t at = 0;        // K and V tiles gone by; a K tile is entry at % R of the ring, its V tile the next
  uint32_t tiles = 0;     // cached tiles gone by
  uint32_t done[NT] = {};  // of them, those that query tile i took part in
  const int role = warp - 4 * NT;  // < 0: softmax

  // Of the unit at hand: its kv-head, first query, and how many query tiles it has; the highest position of a query.
  const auto first_of = [&]() { return by_magic(w.h, p.part.h_magic) * C::kRows; };
  const auto head_of = [&]() { return w.h - by_magic(w.h, p.part.h_magic) * kv.Hkv; };
  const auto tiles_of = [&]() { return NT == 2 && w.u.r.len * p.G - first_of() > 128 ? 2 : 1; };
  const auto highest = [&]() { return p.window > 0 ? load(&part_recs(p.part)[w.n].hi) : 0; };
  // Some query may not see some token of [b, b + kTN).  (A row has one unit of a kv-head, so its first query is `lo`'s.)
  const auto in_part_of = [&](int b, int hi) { return in_part(p, b, w.u.lo, hi); };

  if (role < 0) {
    // ---- softmax: a thread per query ----
    const int tile = warp >> 2, row = tid & 127;
    const float sl2 = p.scale * 1.4426950408889634f;
    uint8_t* qt = smem + tile * C::kQ;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t o_col = lane_base + C::kO + tile * D;
    uint32_t chk = 0;   // parity of checked, a bit per ring phase
    uint32_t mine = 0;  // cached tiles that this query tile took part in
    // Brings the unit's queries to shared memory.  (No product reads those of the unit before any more once its last
    // scores are ready.)
    const auto begin = [&]() {
      if (!w.valid() || tile >= tiles_of()) return;
      const int qi = first_of() + tile * 128 + row;
      const bool there = qi < w.u.r.len * p.G;
      const int t = by_magic(qi, p.part.g_magic);  // token of the part
      int g = -1;
      if (there) g = kv_token(p.rows, w.u.r.bos + t, p.num_global, p.status);
      const int64_t head = (int64_t)(head_of() * p.G + (there ? qi - t * p.G : 0)) * D;
      load_queries<D>(p, qt, 32 * (warp & 3), g >= 0 ? (int64_t)g * p.q_stride + head : -1);
      tc::fence_async_smem();
      tc::mbar_arrive(&sm.q_ready[tile]);
    };
    begin();
    while (w.valid() && ok) {
      const int hi = highest();
      if (tile >= tiles_of()) {
        for (int j = w.j0; j < w.j0 + w.len; ++j, ++tiles)
          if (in_part_of(w.tile_at(j), hi)) chk ^= 1u << (tiles % kPh);
        w.next();
        begin();
        continue;
      }
      const int qi = first_of() + tile * 128 + row;
      const bool there = qi < w.u.r.len * p.G;
      const int t = by_magic(qi, p.part.g_magic);
      // (without a window it does not matter how far behind a group's part its queries stand)
      const int pos = p.window > 0 && there ? load(&part_tokens(p.part)[w.u.r.bos + t].x)
                                            : min(w.u.lo + t, w.u.r.kv - 1);
      float m = -INFINITY, l = 0.f;  // the maximum that the weights refer to (of scores before their scale); their
                                     // sum, both l's and O's 2^-kGrow of e^(s - m)'s
      bool wrote = false;            // O holds something, or will
      for (int j = w.j0; j < w.j0 + w.len; ++j, ++tiles, ++mine) {
        const uint32_t buf = mine & 1, phase = tiles % kPh;
        const uint32_t s_col = lane_base + tile * 128 + buf * 64;
        const int b = w.tile_at(j);
        // O is complete when the product of the tile before is.
        const auto o_complete = [&]() {
          const uint32_t last = mine - 1;
          ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&sm.pv_done[tile][buf ^ 1], (last >> 1) & 1, P.wait_ns));
          tc::fence_after();
          return ok;
        };
        ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&sm.s_ready[tile][buf], (mine >> 1) & 1, P.wait_ns));
        if (!ok) break;
        tc::fence_after();
        uint32_t r[2][32];
        ld_begin(s_col, r[0]);
        ld_begin(s_col + 32, r[1]);
        const uint32_t have = sm.held[tiles & 15];
        const bool all_pages = have == (1u << boxes) - 1u;
        const bool look = in_part_of(b, hi);
        ld_wait(r[0]);
        ld_wait(r[1]);
        if (!all_pages || look) {
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
        const float ms = m == -INFINITY ? 0.f : fmaf(-m, sl2, -kGrow);  // so that no weight passes 1
        const uint64_t scale = pair(sl2, sl2), shift2 = pair(ms, ms);
        uint64_t sum[2] = {0, 0};
        if constexpr (PAIR) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float u[16], low[16];
            weights32<true>(r[i], scale, shift2, sum, u, low);
            tc::tmem_st16(s_col + 16 * i, u);
            tc::tmem_st16(s_col + 32 + 16 * i, low);
          }
        } else {
          float u[32];
          weights32(r[0], scale, shift2, sum, u);
          weights32(r[1], scale, shift2, sum, u + 16);
          tc::tmem_st32(s_col, u);
        }
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
            add_listed<D, PAIR>(p, w.u.r.trow, head_of(), sm.bad[phase], b, pos, s_col, o_col);
          }
        }
        tc::fence_before();
        tc::mbar_arrive(&sm.p_ready[tile][buf]);
        wrote = true;
      }
      if (!ok) break;
      // where this piece goes
      const bool whole = w.j0 == 0 && w.len == w.u.tiles;
      const int64_t place = ((int64_t)(w.n < p.part.groups ? 0 : p.part.tokens) + w.u.r.bos + t) * p.Hq +
                            head_of() * p.G + qi - t * p.G;
      const int slot = 2 * blockIdx.x + (w.j0 == 0 ? 1 : 0), at_tile = tile * 128 + row;
      const int64_t to = whole ? place : (int64_t)slot * C::kRows + at_tile;
      if (there && w.j0 == 0)
        p.part.range[place] = {whole ? -1 : (int)blockIdx.x, whole ? 0 : sm.deal.owner(w.unit_last(sm.share)), tile * 128 + row, 0};
      w.next();
      begin();  // the next unit's first scores come up while O goes out
      const uint32_t last = mine - 1;
      ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&sm.pv_done[tile][last & 1], (last >> 1) & 1, P.wait_ns));
      if (!ok) break;
      tc::fence_after();
      if (there) *reinterpret_cast<float2*>((whole ? p.part.ml : P.stats) + to * 2) = make_float2(m, l);
      // four columns of all queries side by side: a warp's store goes to 512 bytes in a row, not to 32 places (3 us a unit)
      const int64_t step = whole ? (int64_t)2 * p.part.tokens * p.Hq : C::kRows;
      float4* dst = reinterpret_cast<float4*>(whole ? p.part.o : P.o) + (whole ? place : (int64_t)slot * (D / 4) * C::kRows + at_tile);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        tc::tmem_ld32(o_col + c, o);
        if (there) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[(c / 4 + i) * step] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      // The next unit's first product overwrites O; its p_ready, which this thread arrives at, comes after these loads.
    }
    if (!ok) set_status(p.status, GDN_STATUS_WAIT_TIMEOUT);
  } else if (role <= 1) {
    // ---- products: a lane of warp 0 issues all S = Q K^T, one of warp 1 all O += P V ----
    const uint32_t base = tc::smem_addr(smem);
    uint32_t chk = 0;          // parity of checked, a bit per ring phase
    uint32_t units[NT] = {};   // units that query tile i took part in
    // (a phase of a barrier; false once a wait has given up)
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && tc::mbar_wait(bar, parity & 1, P.wait_ns);
      if (ok) tc::fence_after();
      return ok;
    };
    for (; w.valid() && ok; w.next()) {
      const int n = w.len, nt = tiles_of(), hi = highest();
      if (lane == 0 && role == 0) {
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t t = tiles + j, phase = t % kPh;
          if (!wait(&sm.full[2 * phase], t / kPh)) break;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            if (i >= nt) continue;
            const uint32_t d = done[i] + j, buf = d & 1;
            if (j == 0 && !wait(&sm.q_ready[i], units[i])) break;
            // the buffer is free once the product two tiles before is done
            if (d >= 2 && !wait(&sm.pv_done[i][buf], (d >> 1) - 1)) break;
            s_products<D>(base, i, phase, i * 128 + buf * 64);
            tc::commit(&sm.s_ready[i][buf]);
          }
          tc::commit(&sm.empty[2 * phase]);
        }
      } else if (lane == 0) {
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t t = tiles + j, phase = t % kPh;
          bool onto = j > 0;  // O holds listed tokens' share by then
          if (!wait(&sm.full[2 * phase + 1], t / kPh)) break;
          if (in_part_of(w.tile_at(w.j0 + j), hi)) {
            if (!wait(&sm.checked[phase], chk >> phase)) break;
            chk ^= 1u << phase;
            onto |= (sm.bad[phase][0] | sm.bad[phase][1]) != 0;
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            if (i >= nt) continue;
            const uint32_t d = done[i] + j, buf = d & 1;
            if (!wait(&sm.p_ready[i][buf], d >> 1)) break;
            pv_products<D, PAIR>(base, i, phase, i * 128 + buf * 64, onto);
            tc::commit(&sm.pv_done[i][buf]);
          }
          tc::commit(&sm.empty[2 * phase + 1]);
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      tiles += n;
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (i < nt) {
          done[i] += n;
          ++units[i];
        }
    }
    if (lane == 0) {
      tc::commit(&sm.drain[role]);
      if (!tc::mbar_wait(&sm.drain[role], 0, P.wait_ns)) ok = false;
      if (!ok) set_status(p.status, GDN_STATUS_WAIT_TIMEOUT);
    }
    __syncwarp();
  } else if (role == 2) {
    // ---- fetches: a lane per page of the tile ----
    // With a long ring K's pages and V's go together, a half of the warp each, in half the time (a step of one query tile is
    // short: 64 rows of 8000 own tokens, pages of 16, d = 64, 385 us one after the other, 353 together); with a short one K does
    // not wait for V's place.
    constexpr bool kTogether = kPh > 2;
    const int bi = kTogether ? lane & 15 : lane, spp = slabs_per_page(kv);
    const int none = (kv.num_pages - 1) * spp + kv.Hkv;  // a slab past the pool
    const bool active = bi < boxes;
    uint32_t fetched = 0;  // tiles fetched, K and V
    for (; w.valid() && ok; w.next()) {
      const int32_t* row = kv.table + (int64_t)w.u.r.trow * kv.max_pages;
      const int entries = (w.u.r.kv + ps - 1) >> shift, h = head_of();
      int eb = -64, ids = 0, ahead = 0;  // 32 table entries are held, one per lane, and the 32 behind them
      for (int j = w.j0; j < w.j0 + w.len && ok; ++j, at += 2, ++tiles) {
        if (tiles == (uint32_t)P.stop_tile) {
          ok = false;
          break;
        }
        const int b = w.tile_at(j), pos = b + bi * box, e = b >> shift;
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
        const uint32_t mask = __ballot_sync(0xffffffffu, page > 0) & 0xffffu;
        const int slot = pos & (ps - 1), slab = page > 0 ? page * spp + h : none;
        for (int v = kTogether ? lane >> 4 : 0; v < 2; v += kTogether ? 2 : 1) {
          const uint32_t a = at + v, en = a % R;
          ok = __all_sync(0xffffffffu, a < R || tc::mbar_wait(&sm.empty[en], (a / R - 1) & 1, P.wait_ns));
          if (!ok) break;
          if (lane == 0 && v == 0) sm.held[tiles & 15] = mask;  // (before the arrival, which releases it to those who wait)
          if (bi == 0) tc::expect_tx(&sm.full[en], C::kKv);
          __syncwarp();
          if (active) tc::tma_page(ring + en * C::kKv + bi * box * D * 2, v ? &vmap : &kmap, slot, slab, &sm.full[en]);
          fetched = kTogether ? at + 2 : a + 1;
        }
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
    for (; w.valid() && ok; w.next()) {
      const int hi = highest();
      for (int j = w.j0; j < w.j0 + w.len && ok; ++j, at += 2) {
        const int b = w.tile_at(j);
        const uint32_t en = (at + 1) % R;
        const bool look = in_part_of(b, hi);
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
          const bool past = b + t >= w.u.r.kv;
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

template <int D, bool PAIR>
cudaError_t launch_d(const AttnLaunch& a, cudaStream_t s) {
  using C = Cfg<D>;
  static std::atomic<uint64_t> done{0};
  constexpr int smem = (int)(C::kTiles * C::kQ + 2 * phases_of(D) * C::kKv + sizeof(Small<D>));
  static_assert(smem <= 232448, "shared memory");
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(shared_kernel<D, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap kmap, vmap;
  if (!encode_pool_maps(a.cache, a.cache.page_size < kTN ? a.cache.page_size : kTN, &kmap, &vmap))
    return cudaErrorInvalidValue;
  SharedParams P{};
  P.a = a;
  const PartPieces pieces = attn_shared_pieces(a, a.ws);
  P.stats = pieces.stats;
  P.o = pieces.o;
  const uint64_t wait = g_test_wait_ns.load(std::memory_order_relaxed);
  P.wait_ns = wait ? wait : kDefaultWaitNs;
  P.stop_tile = g_test_stop_tile.load(std::memory_order_relaxed);
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
  return cudaLaunchKernelEx(&cfg, shared_kernel<D, PAIR>, P, kmap, vmap);
}

template <bool PAIR>
cudaError_t launch_any(const AttnLaunch& a, cudaStream_t s) {
  return a.cache.d == 64    ? launch_d<64, PAIR>(a, s)
         : a.cache.d == 128 ? launch_d<128, PAIR>(a, s)
                            : launch_d<256, PAIR>(a, s);
}

int rows_of_cta(const AttnLaunch& a) { return a.cache.d <= 128 ? Cfg<128>::kRows : Cfg<256>::kRows; }

}  // namespace

bool attn_shared_supported(const AttnLaunch& a, gdn_dtype dtype) {
  return attn_prompt_supported(a, dtype) && (int64_t)a.rows.max_q * a.G <= rows_of_cta(a);
}

size_t attn_shared_workspace(const AttnLaunch& a) { return (size_t)2 * kSms * rows_of_cta(a) * (a.cache.d + 2) * 4; }

PartPieces attn_shared_pieces(const AttnLaunch& a, void* ws) {
  const int rows = rows_of_cta(a);
  float* stats = static_cast<float*>(ws);
  return {stats, stats + (size_t)4 * kSms * rows, rows, kSms};
}

// Two terms a weight wherever attention without groups would take some row of the call to the split kernel, which keeps 16 bits.
cudaError_t launch_attn_shared(const AttnLaunch& a, cudaStream_t s) {
  const bool pair = attn_split_supported(a, GDN_BF16) || attn_few(a, GDN_BF16) > 0;
  return pair ? launch_any<true>(a, s) : launch_any<false>(a, s);
}

}  // namespace gdn

extern "C" int gdn_testing_set_shared_faults(uint64_t wait_ns, int32_t stop_tile) {
  gdn::g_test_wait_ns.store(wait_ns, std::memory_order_relaxed);
  gdn::g_test_stop_tile.store(stop_tile < 0 ? -1 : stop_tile, std::memory_order_relaxed);
  return GDN_OK;
}
