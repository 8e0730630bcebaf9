// gdn_attn_share.cuh -- rows split over the cache's length: who works on what, and how pieces meet.
//
// A unit is one (row, kv-head), or one group of a row's queries of a kv-head: the 32-token tiles that
// its queries see, window and first tokens included, and kStart tiles in front that stand for what beginning a
// unit takes.  All units' tiles laid end to end are dealt out evenly to the workers.  A share's piece of a unit that
// is not the whole unit leaves (m, l, o) in the workspace; join_kernel adds a unit's pieces in the order of the
// workers.
//
// PART: a pass over parts of the rows' caches, listed as PartRec: a group's queries over what its rows share, a row's over
// its own tokens.  Every query's (m, l, o) over its part comes out, whole or in pieces, and where they are; the join of
// parts (gdn_attn_parts.cu) makes the outputs.
#pragma once

#include <algorithm>

#include "gdn_attn_plan.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace split {

constexpr int kTN = 32;       // tokens of a tile
// Beginning a unit takes about as long as 2 to 3 tiles: without them in the deal, of 64 decode rows' workers those
// with pieces of one unit took 107 thousand cycles, of three 121 and of four 133.
constexpr int kStart = 2;
constexpr int kJoinWarps = 8;
constexpr int kJoinBlocks = 16 * kSms;  // of a launch, more only where the queries need them

struct SplitParams {
  AttnLaunch a;
  float* part;     // [2 * workers][queries of a unit][D]
  float* stats;    // [2 * workers][queries of a unit][2]: m (of the scores before their scale), l
  int32_t* info;   // [workers][8]: the unit that begins in a worker's share and ends in another's
  uint64_t wait_ns;
};

struct Unit {
  KvRow r;
  int sink_tiles, first_tile, tiles;
  int per;       // units of the row
  int from, lo;  // PART: the part's first token, the lowest position of a query
  __device__ int cost(int start) const { return tiles > 0 ? tiles + start : 0; }
};

// A row's values as they lie in memory; with PART, a part's.
template <bool PART>
struct RawRow {
  int bos, eos, kv, trow;
};
template <>
struct RawRow<true> {
  int bos, len, from, end, trow, lo;
};
template <bool PART>
__device__ __forceinline__ int rows_of(const AttnLaunch& p) {
  return PART ? p.part.count : p.rows.num_seqs;
}
// near: the parts in shared memory, if they are there.
template <bool PART>
__device__ __forceinline__ RawRow<PART> raw_row(const AttnLaunch& p, int n, const PartRec* near = nullptr) {
  if constexpr (PART) {
    if (near) return {near[n].bos, near[n].len, near[n].from, near[n].end, near[n].trow, near[n].lo};
    const int4* rec = reinterpret_cast<const int4*>(part_recs(p.part) + n);
    const int4 a = load(rec), b = load(rec + 1);
    return {a.x, a.y, a.z, a.w, b.x, b.y};
  } else {
    return {load(p.rows.qsl + n), load(p.rows.qsl + n + 1), load(p.rows.kv_lens + n),
            p.rows.table_rows ? load(p.rows.table_rows + n) : n};
  }
}
template <bool PART>
__device__ __forceinline__ RawRow<PART> raw_of_lane(const RawRow<PART>& r, int src) {
  const auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
  if constexpr (PART)
    return {of(r.bos), of(r.len), of(r.from), of(r.end), of(r.trow), of(r.lo)};
  else
    return {of(r.bos), of(r.eos), of(r.kv), of(r.trow)};
}

// The tiles that the row's queries see; 0 for an empty or bad row.  QG: queries of a unit, 0 for all
// of a row and kv-head.
template <int QG, bool PART, int TN>
__device__ __forceinline__ Unit unit_of(const AttnLaunch& p, const RawRow<PART>& r, uint32_t* st) {
  Unit u;
  u.tiles = u.sink_tiles = u.first_tile = 0;
  u.per = p.cache.Hkv;
  if constexpr (PART) {
    u.r = KvRow{r.bos, r.len, r.end, r.trow};
    u.from = r.from;
    u.lo = r.lo;
    if (r.len == 0) return u;
    const int tokens = r.end - r.from;
    const int low = p.window > 0 ? min(max(max(0, r.lo - p.window + 1) - r.from, 0), tokens) : 0;
    u.sink_tiles = (min(max(p.sinks - r.from, 0), low) + TN - 1) / TN;
    u.first_tile = max(low / TN, u.sink_tiles);
    u.tiles = u.sink_tiles + max((tokens + TN - 1) / TN - u.first_tile, 0);
    u.per *= (int)(((int64_t)r.len * p.G + QG - 1) / QG);
    return u;
  } else {
    if (!check_kv_row(p.rows, p.cache, r.bos, r.eos, r.kv, r.trow, u.r, st) || u.r.len == 0 ||
        (p.few > 0 && u.r.len * p.G > p.few))
      return u;
    const int low = p.window > 0 ? max(0, u.r.kv - u.r.len - p.window + 1) : 0;
    u.sink_tiles = (min(p.sinks, low) + kTN - 1) / kTN;
    u.first_tile = max(low / kTN, u.sink_tiles);
    u.tiles = u.sink_tiles + (u.r.kv + kTN - 1) / kTN - u.first_tile;
    if (QG > 0) u.per *= (u.r.len * p.G + QG - 1) / (QG > 0 ? QG : 1);
    return u;
  }
}
// The cost in tiles of all units of row n.
template <int QG, bool PART, int TN>
__device__ __forceinline__ int64_t row_cost(const AttnLaunch& p, int n, int start, uint32_t* st, const PartRec* near) {
  const Unit u = unit_of<QG, PART, TN>(p, raw_row<PART>(p, n, near), st);
  return (int64_t)u.cost(start) * u.per;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The tiles dealt to the workers: the first `more` get each + 1, the others each.
struct Deal {
  int64_t each;
  int more;
  int start;  // tiles that a unit's beginning counts
  __device__ int64_t first(int worker) const { return each * worker + min(worker, more); }
  __device__ int owner(int64_t tile) const;
};

// 64-bit quotient; in 32 bits where that does.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int Deal::owner(int64_t tile) const {
  const int64_t head = (each + 1) * more;
  return (int)(tile < head ? quotient(tile, each + 1) : more + quotient(tile - head, each));
}

// A worker's share of the tiles, and where it begins.
template <bool PART>
struct Share {
  int64_t first;
  int64_t into;  // tiles of row `row` before the share
  int row;
  int span;      // tiles
  RawRow<PART> raw;  // that row
};

// The shares of the CTA's workers; part: one value per warp; near: the parts in shared memory, if they are there.  A unit's
// beginning counts START tiles, or HALF where no unit has more than half of QG queries.  All threads call.
template <int QG, int NW, int THREADS, bool PART = false, int TN = kTN, int START = kStart, int HALF = START>
__device__ void find_shares(const AttnLaunch& p, int64_t* part, Deal& deal, Share<PART>* shares,
                            const PartRec* near = nullptr) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = rows_of<PART>(p), per = (rows + THREADS - 1) / THREADS;
  const int n0 = min(tid * per, rows), n1 = min(n0 + per, rows);
  int64_t mine = 0;
  int start = START;
  if constexpr (HALF != START) {
    int64_t units = 0;
    bool full = false;
    for (int n = n0; n < n1; ++n) {
      const Unit u = unit_of<QG, PART, TN>(p, raw_row<PART>(p, n, near), nullptr);
      if (u.tiles == 0) continue;
      mine += (int64_t)u.tiles * u.per;
      units += u.per;
      full |= (int64_t)u.r.len * p.G > QG / 2;
    }
    if (!__syncthreads_or(full)) start = HALF;
    mine += units * start;
  } else {
    for (int n = n0; n < n1; ++n) mine += row_cost<QG, PART, TN>(p, n, START, blockIdx.x == 0 ? p.status : nullptr, near);
  }
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int64_t before = inc - mine, total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) before += part[i];
    total += part[i];
  }
  Deal d;
  const int workers = gridDim.x * NW;
  d.each = quotient(total, workers);
  d.more = (int)(total - d.each * workers);
  d.start = start;
  if (tid == 0) deal = d;
#pragma unroll 1
  for (int w = 0; w < NW; ++w) {
    Share<PART> s;
    s.first = d.first(blockIdx.x * NW + w);
    s.span = (int)(d.first(blockIdx.x * NW + w + 1) - s.first);
    s.row = 0;
    s.into = 0;
    s.raw = RawRow<PART>{};
    if (s.span == 0) {
      if (tid == 0) shares[w] = s;
    } else if (s.first >= before && s.first < before + mine) {  // one thread
      int64_t at = before;
      int n = n0;
      if (per > 1) {
        for (; n < n1; ++n) {
          const int64_t t = row_cost<QG, PART, TN>(p, n, start, nullptr, near);
          if (s.first < at + t) break;
          at += t;
        }
      }
      s.row = n;
      s.into = s.first - at;
      s.raw = raw_row<PART>(p, n, near);
      shares[w] = s;
    }
  }
  tc::fence_async_smem();  // `part` is memory that copies write next
  __syncthreads();
}

// Walks the units of a share: (row, unit of the row, tiles [j0, j0 + len) of the unit).  A warp holds the raw
// values of the next 32 rows, one per lane, so that going on to the next row waits for no memory.
// All lanes call together.
template <int QG, bool PART = false, int TN = kTN>
struct Walk {
  const AttnLaunch& p;
  const int start;  // the deal's
  int left;
  int n, h, j0, len;  // h: unit of the row
  Unit u;
  __device__ Walk(const AttnLaunch& launch, const Share<PART>& s, int start_ = kStart)
      : p(launch), start(start_), left(s.span), n(s.row), len(0) {
    if (left <= 0) return;
    fill(n + 1);
    u = unit_of<QG, PART, TN>(p, s.raw, nullptr);
    h = (int)quotient(s.into, u.cost(start));
    piece((int)(s.into - (int64_t)h * u.cost(start)));
  }
  __device__ bool valid() const { return left > 0; }
  __device__ void next() {
    left -= span;
    if (left <= 0) return;
    if (++h == u.per) {
      h = 0;
      do {
        if (++n >= rows_of<PART>(p)) {
          left = 0;
          return;
        }
        if (n == base + 32) fill(n);
        u = unit_of<QG, PART, TN>(p, raw_of_lane<PART>(ahead, n - base), nullptr);
      } while (u.tiles == 0);
    }
    piece(0);
  }
  __device__ int tile_at(int j) const {
    const int at = (j < u.sink_tiles ? j : u.first_tile + j - u.sink_tiles) * TN;
    return PART ? u.from + at : at;
  }
  // Where the unit ends in the deal.
  __device__ int64_t unit_last(const Share<PART>& s) const { return s.first + s.span - left - from + u.cost(start) - 1; }

 private:
  int from, span;  // the piece in the unit's tiles with those that stand for its beginning
  __device__ void piece(int at) {
    from = at;
    span = min(u.cost(start) - at, left);
    j0 = max(at - start, 0);
    len = at + span - start - j0;
    if (len <= 0) left = 0;  // the share ends before the unit's first tile
  }
  int base;
  RawRow<PART> ahead;
  __device__ void fill(int from) {
    base = from;
    ahead = raw_row<PART>(p, min(from + (int)(threadIdx.x & 31), rows_of<PART>(p) - 1));
  }
};

// Adds the pieces of the unit that begins in worker blockIdx.x's share and ends in a later one's.  A warp per query, or
// a team of them; a lane per piece for the statistics, then eight pieces' values on their way at a time; the blocks
// of a column share the queries.  (A block per CTA of the attention, which took its workers' units and their
// pieces in turn, took 16 us under 128 windowed verify rows; that call went from 59.6 us to 52.7.)
inline int join_rows(int workers, int queries) {
  return std::max((queries + kJoinWarps - 1) / kJoinWarps, std::min(queries, std::min(kJoinWarps, kJoinBlocks / workers)));
}
// E: 32 E columns or fewer are worked on; DC: head_dim, 0 for that of the cache.
template <typename T, int E, int DC>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(SplitParams P, int queries) {
  __shared__ float so[kJoinWarps][32 * E];
  __shared__ float sl[kJoinWarps], sm[kJoinWarps];
  const AttnLaunch& p = P.a;
  const float sl2 = p.scale * 1.4426950408889634f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kAtOnce = 8;  // pieces whose values are on their way
  const int D = DC > 0 ? DC : p.cache.d;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c0 = blockIdx.x, f = lane < 8 ? P.info[c0 * 8 + lane] : 0;
  if (__shfl_sync(0xffffffffu, f, 0)) {
    const int bos = __shfl_sync(0xffffffffu, f, 1), nq = __shfl_sync(0xffffffffu, f, 2);
    const int h = __shfl_sync(0xffffffffu, f, 3), c1 = __shfl_sync(0xffffffffu, f, 4);
    const int qi0 = __shfl_sync(0xffffffffu, f, 5);  // the unit's first query
    const int pieces = c1 - c0 + 1;
    const int team = pieces > 64 ? 8 : pieces > 32 ? 4 : pieces > 16 ? 2 : 1;  // warps of a query
    for (int q0 = blockIdx.y * (kJoinWarps / team); q0 < nq; q0 += gridDim.y * (kJoinWarps / team)) {
      const int qi = q0 + warp / team;
      float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
      for (int i = 0; i < E; ++i) o[i] = 0.f;
      if (qi < nq) {
        const int mine = (pieces - warp % team + team - 1) / team;  // this warp's pieces: every team-th
        for (int s0 = 0; s0 < mine; s0 += 32) {
          // a lane per piece for the statistics
          auto place = [&](int i) {
            const int c = c0 + warp % team + team * (s0 + i);
            return (size_t)(2 * c + (c == c0 ? 1 : 0)) * queries + qi;
          };
          const float2 st = s0 + lane < mine ? *reinterpret_cast<const float2*>(P.stats + place(lane) * 2)
                                             : make_float2(-INFINITY, 0.f);
          float mn = st.x;
#pragma unroll
          for (int d = 16; d; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
          mn = fmaxf(mn, m);
          const float a = m == -INFINITY ? 0.f : ex2((m - mn) * sl2);
          const float f = st.x == -INFINITY ? 0.f : ex2((st.x - mn) * sl2);
          float sum = st.y * f;
#pragma unroll
          for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          l = l * a + sum;
          m = mn;
#pragma unroll
          for (int i = 0; i < E; ++i) o[i] *= a;
          for (int u0 = 0; u0 < 32 && s0 + u0 < mine; u0 += kAtOnce) {
            float v[kAtOnce][E];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
              for (int i = 0; i < E; ++i)
                v[u][i] = s0 + u0 + u < mine && (DC > 0 || lane + 32 * i < D) ? P.part[place(u0 + u) * D + lane + 32 * i] : 0.f;
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
              const float b = __shfl_sync(0xffffffffu, f, u0 + u);
#pragma unroll
              for (int i = 0; i < E; ++i) o[i] = fmaf(v[u][i], b, o[i]);
            }
          }
        }
      }
      if (team > 1) {
#pragma unroll
        for (int i = 0; i < E; ++i) so[warp][lane + 32 * i] = o[i];
        if (lane == 0) {
          sm[warp] = m;
          sl[warp] = l;
        }
        __syncthreads();
        if (warp % team == 0) {
          for (int v = warp + 1; v < warp + team; ++v) {
            const float mn = fmaxf(m, sm[v]);
            const float a = m == -INFINITY ? 0.f : ex2((m - mn) * sl2);
            const float b = sm[v] == -INFINITY ? 0.f : ex2((sm[v] - mn) * sl2);
            l = l * a + sl[v] * b;
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = o[i] * a + so[v][lane + 32 * i] * b;
            m = mn;
          }
        }
        __syncthreads();
      }
      if (qi >= nq || warp % team) continue;
      const int t = (qi0 + qi) / p.G;
      const int g = p.rows.tok ? load(p.rows.tok + bos + t) : bos + t;
      if (g < 0 || g >= p.num_global) continue;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      T* out = static_cast<T*>(p.out) + (int64_t)g * p.out_stride + (int64_t)(h * p.G + qi0 + qi - t * p.G) * D;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (DC > 0 || lane + 32 * i < D) out[lane + 32 * i] = from_f32<T>(o[i] * inv);
    }
  }
}

}  // namespace split
}  // namespace gdn
