// gdn_kv_pages.cu -- the pages of the key-value cache: append, reserve, release, fork, copy, compact.
//
// State on the device: the block table and refcount[p], the number of table entries that hold
// page p.  There is no free list to keep in step with them: a page is free when its count is 0,
// and pages are handed out lowest id first, so every call is a function of the table and the
// counts alone.  Handing out is three steps:
//   count:  per row the pages it needs; per block of pages how many are free;
//   list:   the free pages, lowest first, up to the total need, and the rows' exclusive sums;
//   assign: row i takes free[offset_i ..] when offset_i + need_i is covered.
// Pools of up to 131072 pages (kHandPages) go through them in one launch of a cluster, with barriers in
// between; larger ones, and forks in tables of long rows (kHandEntries), in three dependent launches.
// Counters change by integer adds only, so their order does not matter.
#include "gdn_kv.cuh"

namespace gdn {

namespace {

constexpr int kPageBlock = 1024;  // pages counted by one block
constexpr int kThreads = 256;
constexpr int kPer = kPageBlock / kThreads;

__host__ __device__ inline int page_blocks(int32_t num_pages) { return (num_pages + kPageBlock - 1) / kPageBlock; }

__host__ __device__ inline int max_of(int a, int b) { return a > b ? a : b; }

// Workspace, in ints: need[count] | off[count] | old[count] | fresh[count] | used[count] |
// blocks[page_blocks, at least 8] | total[4] | list_a[num_pages] | list_b[num_pages].
struct Ws {
  int32_t *need, *off, *old_page, *new_page, *used, *blocks, *total, *list_a, *list_b;
};
__host__ __device__ inline Ws carve(int32_t* w, int32_t num_pages, int32_t count) {
  Ws s;
  s.need = w;
  s.off = s.need + count;
  s.old_page = s.off + count;
  s.new_page = s.old_page + count;
  s.used = s.new_page + count;
  s.blocks = s.used + count;
  s.total = s.blocks + max_of(page_blocks(num_pages), 8);
  s.list_a = s.total + 4;
  s.list_b = s.list_a + num_pages;
  return s;
}

__device__ __forceinline__ void wait_prior() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Sum over the block; every thread gets it.  kThreads threads.
__device__ int block_sum(int v) {
  __shared__ int part[kThreads / 32];
  __shared__ int all;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    int t = 0;
    for (int i = 0; i < kThreads / 32; ++i) t += part[i];
    all = t;
  }
  __syncthreads();
  return all;
}

// Exclusive sum over the block's threads; `total` is the whole.  kThreads threads.
__device__ int block_scan(int v, int& total) {
  __shared__ int part[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += part[i];
    total += part[i];
  }
  __syncthreads();
  return before + inc - v;
}

__device__ __forceinline__ bool free_page(const KvDev& C, int p) { return p > 0 && p < C.num_pages && C.refcount[p] == 0; }
__device__ __forceinline__ bool live_page(const KvDev& C, int p) { return p > 0 && p < C.num_pages && C.refcount[p] > 0; }

// ---- append -----------------------------------------------------------------------------------

constexpr int kHeld = 4;  // 16-byte vectors of K and of V that a lane holds

// A warp per token: 16-byte vectors over the token's Hkv x d elements, read and written once: HBM bounds it.  The
// token's values are on their way before its page is looked up, which takes four loads one after another (8192
// tokens of 8 kv-heads, d = 128: 12.5 us = 5.4 TB/s; looked up first, 20.3).
__global__ void __launch_bounds__(kThreads) append_kernel(AppendLaunch p) {
  const KvDev& C = p.cache;
  let_next();
  wait_prior();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int local = blockIdx.x * (kThreads / 32) + warp;
  if (local >= p.rows.num_tokens) return;
  const int32_t g = p.rows.tok ? load(p.rows.tok + local) : local;
  const bool there = g >= 0 && g < p.num_global;
  const int vec = C.d * p.es / 16;  // 16-byte vectors of one head
  const int all = C.Hkv * vec;
  const uint4* ks = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.k) + (int64_t)g * p.k_stride * p.es);
  const uint4* vs = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.v) + (int64_t)g * p.v_stride * p.es);
  uint4 kx[kHeld], vx[kHeld];
  auto fetch = [&](int from) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int i = from + 32 * u + lane;
      kx[u] = there && i < all ? load(ks + i) : make_uint4(0, 0, 0, 0);
      vx[u] = there && i < all ? load(vs + i) : make_uint4(0, 0, 0, 0);
    }
  };
  fetch(0);
  // the row of the token: the last one that begins at or before it
  int lo = 0, hi = p.rows.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (load(p.rows.qsl + mid) <= local) lo = mid; else hi = mid - 1;
  }
  KvRow r;
  if (!load_kv_row(p.rows, C, lo, r, p.status) || local < r.bos || local >= r.bos + r.len) return;
  const int pos = r.kv - r.len + (local - r.bos);
  const int32_t raw = C.table[(int64_t)r.trow * C.max_pages + pos / C.page_size];
  const int32_t page = page_or_null(raw, C, p.status);
  if (page == 0) return;
  if (C.refcount && C.refcount[page] > 1) {
    set_status(p.status, GDN_STATUS_PAGE_SHARED);
    return;
  }
  if (!there) {
    set_status(p.status, GDN_STATUS_TOKEN_RANGE);
    return;
  }
  const int slot = pos % C.page_size, by = __ffs(vec) - 1;
  const int64_t page_off = (int64_t)page * C.page_stride * p.es;
  uint4* kd = reinterpret_cast<uint4*>(static_cast<uint8_t*>(C.k) + page_off);
  uint4* vd = reinterpret_cast<uint4*>(static_cast<uint8_t*>(C.v) + page_off);
  const bool shift = (vec & (vec - 1)) == 0;
  for (int from = 0; from < all; from += 32 * kHeld) {
    if (from > 0) fetch(from);
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int i = from + 32 * u + lane;
      if (i >= all) break;
      const int h = shift ? i >> by : i / vec, c = i - h * vec;
      const int64_t o = ((int64_t)h * C.page_size + slot) * vec + c;
      kd[o] = kx[u];
      vd[o] = vx[u];
    }
  }
}

// ---- handing out pages --------------------------------------------------------------------------

struct RowNeed {
  int trow, lo, hi;  // reserve: entries [lo, hi) of the table row
};

__device__ bool reserve_range(const PageRowsLaunch& p, int i, RowNeed& r) {
  const KvDev& C = p.cache;
  r.trow = p.rows ? load(p.rows + i) : i;
  const int from = load(p.a + i), to = load(p.b + i);
  if (r.trow < 0 || r.trow >= C.num_table_rows || from < 0 || to < 0 ||
      (int64_t)to > (int64_t)C.max_pages * C.page_size)
    return false;
  r.lo = (int)(((int64_t)from + C.page_size - 1) / C.page_size);
  r.hi = (int)(((int64_t)to + C.page_size - 1) / C.page_size);
  return true;
}

// Fork i: whether it can be done, its shared entries, its partly filled page (0 = none).
struct ForkItem {
  int src, dst, full, part;
};
__device__ bool fork_item(const PageRowsLaunch& p, int i, ForkItem& f) {
  const KvDev& C = p.cache;
  f.src = load(p.src_rows + i);
  f.dst = load(p.rows + i);
  const int len = load(p.a + i);
  if (f.src < 0 || f.src >= C.num_table_rows || f.dst < 0 || f.dst >= C.num_table_rows || len < 0 ||
      (int64_t)len > (int64_t)C.max_pages * C.page_size)
    return false;
  f.full = len / C.page_size;
  f.part = len % C.page_size;
  return true;
}

// Blocks [0, page_blocks): free pages of a block of pages.  Blocks behind them: a row's need
// (reserve: its empty entries; fork: 1 for a partly filled page; -1 marks a row to skip).
template <bool kFork>
__global__ void __launch_bounds__(kThreads) need_kernel(PageRowsLaunch p) {
  const KvDev& C = p.cache;
  const Ws w = carve(p.ws, C.num_pages, p.count);
  const int nb = page_blocks(C.num_pages);
  let_next();
  wait_prior();
  if ((int)blockIdx.x < nb) {
    const int p0 = blockIdx.x * kPageBlock;
    int n = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) n += free_page(C, p0 + j * kThreads + threadIdx.x) ? 1 : 0;
    n = block_sum(n);
    if (threadIdx.x == 0) w.blocks[blockIdx.x] = n;
    return;
  }
  const int i = blockIdx.x - nb;
  if (!kFork) {
    RowNeed r;
    if (!reserve_range(p, i, r)) {
      if (threadIdx.x == 0) {
        set_status(p.status, GDN_STATUS_PAGE_RANGE);
        w.need[i] = -1;
      }
      return;
    }
    const int32_t* row = C.table + (int64_t)r.trow * C.max_pages;
    int n = 0;
    for (int e = r.lo + threadIdx.x; e < r.hi; e += kThreads) n += row[e] <= 0 ? 1 : 0;
    n = block_sum(n);
    if (threadIdx.x == 0) w.need[i] = n;
  } else {
    ForkItem f;
    bool ok = fork_item(p, i, f);
    int held = 0, last = 0;
    if (ok) {
      const int32_t* from = C.table + (int64_t)f.src * C.max_pages;
      const int32_t* to = C.table + (int64_t)f.dst * C.max_pages;
      const int n = f.full + (f.part ? 1 : 0);
      for (int e = threadIdx.x; e < n; e += kThreads) held += (to[e] > 0 || from[e] >= C.num_pages) ? 1 : 0;
      if (f.part) last = from[f.full];
    }
    held = block_sum(held);
    ok = ok && held == 0;
    if (threadIdx.x == 0) {
      if (!ok) set_status(p.status, GDN_STATUS_PAGE_RANGE);
      w.need[i] = ok ? (last > 0 ? 1 : 0) : -1;
      w.old_page[i] = ok && last > 0 ? last : 0;
      w.used[i] = ok ? f.part : 0;
    }
  }
}

// The free pages lowest first (list_a), as many as are needed; the last block sums the needs.
__global__ void __launch_bounds__(kThreads) free_list_kernel(PageRowsLaunch p) {
  const KvDev& C = p.cache;
  const Ws w = carve(p.ws, C.num_pages, p.count);
  const int nb = page_blocks(C.num_pages);
  wait_prior();
  let_next();
  if ((int)blockIdx.x == nb) {
    int base = 0;
    for (int i0 = 0; i0 < p.count; i0 += kThreads) {
      const int i = i0 + threadIdx.x;
      const int n = i < p.count ? max(w.need[i], 0) : 0;
      int total;
      const int at = block_scan(n, total);
      if (i < p.count) w.off[i] = base + at;
      base = min(base + total, 1 << 30);  // needs past every pool stay past it
    }
    int free_pages = 0;
    for (int i = threadIdx.x; i < nb; i += kThreads) free_pages += w.blocks[i];
    free_pages = block_sum(free_pages);
    if (threadIdx.x == 0) w.total[0] = free_pages;
    return;
  }
  int before = 0;
  for (int i = threadIdx.x; i < (int)blockIdx.x; i += kThreads) before += w.blocks[i];
  before = block_sum(before);
  // enough found in the blocks before this one?
  long long need = 0;
  for (int i = threadIdx.x; i < p.count; i += kThreads) need += max(w.need[i], 0);
  const int wanted = block_sum((int)min(need, (long long)(1 << 22)));
  if (before >= wanted && wanted < (1 << 22)) return;
  const int p0 = blockIdx.x * kPageBlock + threadIdx.x * kPer;
  uint32_t mask = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) mask |= (free_page(C, p0 + j) ? 1u : 0u) << j;
  int total;
  int at = before + block_scan(__popc(mask), total);
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (mask >> j & 1) w.list_a[at++] = p0 + j;
}

__device__ __forceinline__ bool granted(const Ws& w, int i, uint32_t* st) {
  const int need = w.need[i];
  if (need < 0) return false;
  if (w.off[i] + need > w.total[0]) {
    if (threadIdx.x == 0) set_status(st, GDN_STATUS_NO_PAGES);
    return false;
  }
  return true;
}

__global__ void __launch_bounds__(kThreads) reserve_kernel(PageRowsLaunch p) {
  const KvDev& C = p.cache;
  const Ws w = carve(p.ws, C.num_pages, p.count);
  let_next();
  wait_prior();
  const int i = blockIdx.x;
  RowNeed r;
  if (!reserve_range(p, i, r) || w.need[i] <= 0 || !granted(w, i, p.status)) return;
  int32_t* row = C.table + (int64_t)r.trow * C.max_pages;
  int base = w.off[i];
  for (int e0 = r.lo; e0 < r.hi; e0 += kThreads) {
    const int e = e0 + threadIdx.x;
    const bool empty = e < r.hi && row[e] <= 0;
    int total;
    const int at = block_scan(empty ? 1 : 0, total);
    if (empty) {
      const int page = w.list_a[base + at];
      row[e] = page;
      C.refcount[page] = 1;
    }
    base += total;
  }
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kHandCtas = 8, kHandThreads = 1024;
constexpr int kHandPer = 16;  // pages of a thread
constexpr int kHandPages = kHandCtas * kHandThreads * kHandPer;
// Entries of a table row up to which forks go in one launch.  There a warp walks a row's entries and a cluster has 256
// warps, in three launches a block on any SM does.  64 forks of full rows (pages of 16, time on the GPU): of 62 entries
// 17 us in one launch, 14 in three, of 500 27 and 14, of 1000 38 and 14, of 8000 224 and 32; three more launches cost a
// step that is bound by its launches 3 us a call (release, fork and reserve of 64 rows: 20 us, 26).
constexpr int kHandEntries = 1024;

// Exclusive sum over the threads of a CTA of the cluster.
__device__ int hand_scan(int v, int& total, int* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int w = part[lane];
  const int mine = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  return __shfl_sync(0xffffffffu, w - mine, warp) + inc - v;
}

// Reserve, or fork but for the copies, in one launch of a cluster: a warp per row, a thread per kHandPer pages.
// The three launches that it stands for take their time in starts and ends; what is computed is a few microseconds'
// reads.  Release, fork and reserve of 64 rows take 26 to 29 us in eight launches and 20 in four.
template <bool kFork>
__global__ void __cluster_dims__(kHandCtas) __launch_bounds__(kHandThreads, 1) hand_out_kernel(PageRowsLaunch p) {
  __shared__ int part[32];
  const KvDev& C = p.cache;
  const Ws w = carve(p.ws, C.num_pages, p.count);
  const int cta = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const int warp = cta * (kHandThreads / 32) + (tid >> 5);
  constexpr int kWarps = kHandCtas * kHandThreads / 32;
  let_next();
  wait_prior();
  // count: a row's need (-1: the row is left out), and the thread's free pages
  const int per = (C.num_pages + kHandCtas * kHandThreads - 1) / (kHandCtas * kHandThreads);
  const int p0 = (cta * kHandThreads + tid) * per;
  uint32_t mask = 0;
  for (int j = 0; j < per; ++j) mask |= (free_page(C, p0 + j) ? 1u : 0u) << j;
  for (int i = warp; i < p.count; i += kWarps) {
    bool ok;
    int n = 0, held = 0, last = 0, used = 0;
    if constexpr (kFork) {
      ForkItem f;
      ok = fork_item(p, i, f);
      if (ok) {
        const int32_t* from = C.table + (int64_t)f.src * C.max_pages;
        const int32_t* to = C.table + (int64_t)f.dst * C.max_pages;
#pragma unroll 4
        for (int e = lane; e < f.full + (f.part ? 1 : 0); e += 32) held |= to[e] > 0 || from[e] >= C.num_pages;
        if (f.part) last = from[f.full];
        used = f.part;
      }
      ok = ok && !__any_sync(0xffffffffu, held);
      n = last > 0 ? 1 : 0;
    } else {
      RowNeed r;
      ok = reserve_range(p, i, r);
      if (ok) {
        const int32_t* row = C.table + (int64_t)r.trow * C.max_pages;
#pragma unroll 4
        for (int e = r.lo + lane; e < r.hi; e += 32) n += row[e] <= 0 ? 1 : 0;
        n = __reduce_add_sync(0xffffffffu, n);
      }
    }
    if (lane == 0) {
      if (!ok) set_status(p.status, GDN_STATUS_PAGE_RANGE);
      // (as many as the pool has are never free: the sums of 1024 rows stay below 2^27)
      w.need[i] = ok ? min(n, C.num_pages) : -1;
      if (kFork) {
        w.old_page[i] = ok && last > 0 ? last : 0;
        w.used[i] = ok ? used : 0;
      }
    }
  }
  int total;
  const int before = hand_scan(__popc(mask), total, part);
  if (tid == 0) w.blocks[cta] = total;
  cluster_sync();
  // list: as many pages as are needed; every CTA sums the needs, the first writes the rows' offsets
  int first = 0, have = 0;
#pragma unroll
  for (int i = 0; i < kHandCtas; ++i) {
    const int n = __ldcg(w.blocks + i);
    first += i < cta ? n : 0;
    have += n;
  }
  int base = 0;
  for (int i0 = 0; i0 < p.count; i0 += kHandThreads) {
    const int i = i0 + tid;
    int sum;
    const int at = hand_scan(i < p.count ? max(__ldcg(w.need + i), 0) : 0, sum, part);
    if (cta == 0 && i < p.count) w.off[i] = base + at;
    base = min(base + sum, 1 << 30);  // needs past every pool stay past it (here a pool has 2^17 pages at most)
  }
  if (cta == 0 && tid == 0) w.total[0] = have;
  for (int at = first + before; mask && at < base; mask &= mask - 1) w.list_a[at++] = p0 + __ffs(mask) - 1;
  cluster_sync();
  // assign
  for (int i = warp; i < p.count; i += kWarps) {
    const int need = __ldcg(w.need + i), off = __ldcg(w.off + i);
    const bool enough = off + need <= have;
    if (need >= 0 && !enough && lane == 0) set_status(p.status, GDN_STATUS_NO_PAGES);
    const bool ok = need >= 0 && enough;
    if constexpr (kFork) {
      const int page = ok && need > 0 ? __ldcg(w.list_a + off) : 0;
      if (lane == 0) w.new_page[i] = page;
      ForkItem f;
      if (!ok || !fork_item(p, i, f)) continue;
      const int32_t* from = C.table + (int64_t)f.src * C.max_pages;
      int32_t* to = C.table + (int64_t)f.dst * C.max_pages;
      for (int e0 = lane; e0 < f.full; e0 += 128) {
        int id[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) id[u] = e0 + 32 * u < f.full ? max(from[e0 + 32 * u], 0) : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (e0 + 32 * u < f.full) to[e0 + 32 * u] = id[u];
          if (id[u] > 0) atomicAdd(C.refcount + id[u], 1);
        }
      }
      if (f.part && lane == 0) {
        to[f.full] = page;
        if (page > 0) C.refcount[page] = 1;
      }
    } else {
      RowNeed r;
      if (!ok || need == 0 || !reserve_range(p, i, r)) continue;
      int32_t* row = C.table + (int64_t)r.trow * C.max_pages;
      int next = off;
      for (int e0 = r.lo; e0 < r.hi; e0 += 32) {
        const int e = e0 + lane;
        const bool empty = e < r.hi && row[e] <= 0;
        const uint32_t set = __ballot_sync(0xffffffffu, empty);
        if (empty) {
          const int page = __ldcg(w.list_a + next + __popc(set & ((1u << lane) - 1u)));
          row[e] = page;
          C.refcount[page] = 1;
        }
        next += __popc(set);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads) fork_kernel(PageRowsLaunch p) {
  const KvDev& C = p.cache;
  const Ws w = carve(p.ws, C.num_pages, p.count);
  wait_prior();
  let_next();
  const int i = blockIdx.x;
  ForkItem f;
  const bool ok = fork_item(p, i, f) && granted(w, i, p.status);
  const int page = ok && w.need[i] > 0 ? w.list_a[w.off[i]] : 0;
  if (threadIdx.x == 0) w.new_page[i] = page;
  if (!ok) return;
  const int32_t* from = C.table + (int64_t)f.src * C.max_pages;
  int32_t* to = C.table + (int64_t)f.dst * C.max_pages;
  for (int e = threadIdx.x; e < f.full; e += kThreads) {
    const int id = max(from[e], 0);
    to[e] = id;
    if (id > 0) atomicAdd(C.refcount + id, 1);
  }
  if (f.part && threadIdx.x == 0) {
    to[f.full] = page;
    if (page > 0) C.refcount[page] = 1;
  }
}

// The used tokens of each fork's partly filled page: a block per (fork, kv head, K or V).
__global__ void __launch_bounds__(kThreads) fork_copy_kernel(PageRowsLaunch p) {
  const KvDev& C = p.cache;
  const Ws w = carve(p.ws, C.num_pages, p.count);
  let_next();
  wait_prior();
  const int i = blockIdx.x;
  const int dst = w.new_page[i], src = w.old_page[i];
  if (dst <= 0 || src <= 0) return;
  const int64_t head = (int64_t)blockIdx.y * C.page_size * C.d;
  const int n = w.used[i] * C.d * p.es / 16;
  uint8_t* pool = static_cast<uint8_t*>(blockIdx.z ? C.v : C.k);
  const uint4* s = reinterpret_cast<const uint4*>(pool + ((int64_t)src * C.page_stride + head) * p.es);
  uint4* d = reinterpret_cast<uint4*>(pool + ((int64_t)dst * C.page_stride + head) * p.es);
  for (int j = threadIdx.x; j < n; j += kThreads) d[j] = s[j];
}

// ---- release ------------------------------------------------------------------------------------

__global__ void __launch_bounds__(kThreads) release_kernel(PageRowsLaunch p) {
  const KvDev& C = p.cache;
  let_next();
  wait_prior();
  for (int i = blockIdx.y; i < p.count; i += gridDim.y) {
    const int trow = p.rows ? load(p.rows + i) : i;
    const int lo = p.a ? load(p.a + i) : 0, hi = p.b ? load(p.b + i) : C.max_pages;
    if (trow < 0 || trow >= C.num_table_rows || lo < 0 || hi > C.max_pages) {
      if (blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, GDN_STATUS_PAGE_RANGE);
      continue;
    }
    int32_t* row = C.table + (int64_t)trow * C.max_pages;
    for (int e = lo + blockIdx.x * kThreads + threadIdx.x; e < hi; e += gridDim.x * kThreads) {
      const int id = row[e];
      if (id == 0) continue;
      row[e] = 0;
      if (id < 0) continue;
      if (id >= C.num_pages) {
        set_status(p.status, GDN_STATUS_PAGE_RANGE);
      } else if (atomicSub(C.refcount + id, 1) <= 0) {
        atomicAdd(C.refcount + id, 1);
        set_status(p.status, GDN_STATUS_PAGE_RANGE);
      }
    }
  }
}

// ---- compact ------------------------------------------------------------------------------------

__global__ void __launch_bounds__(kThreads) live_kernel(PageRowsLaunch p) {
  const KvDev& C = p.cache;
  const Ws w = carve(p.ws, C.num_pages, 0);
  let_next();
  wait_prior();
  const int p0 = blockIdx.x * kPageBlock;
  int n = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) n += live_page(C, p0 + j * kThreads + threadIdx.x) ? 1 : 0;
  n = block_sum(n);
  if (threadIdx.x == 0) w.blocks[blockIdx.x] = n;
}

// With M live pages in all: mover r (the r-th live page above M) is listed at list_a[r], hole r
// (the r-th free page up to M) at list_a[M' + r] with M' = num_pages / 2, and list_b[page] = r for a
// mover, -1 for any other page.  At most min(M, num_pages - 1 - M) <= num_pages / 2 pages move.
__global__ void __launch_bounds__(kThreads) plan_kernel(PageRowsLaunch p, int32_t* num_live) {
  const KvDev& C = p.cache;
  const Ws w = carve(p.ws, C.num_pages, 0);
  wait_prior();
  let_next();
  const int nb = page_blocks(C.num_pages);
  int before = 0, all = 0;
  for (int i = threadIdx.x; i < nb; i += kThreads) {
    const int n = w.blocks[i];
    all += n;
    if (i < (int)blockIdx.x) before += n;
  }
  before = block_sum(before);
  const int M = block_sum(all);
  // live pages up to M: those of the whole blocks below, and of M's own block
  const int mb = M / kPageBlock;  // the block that holds page M
  int upto = 0;
  for (int i = threadIdx.x; i < mb; i += kThreads) upto += w.blocks[i];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int q = mb * kPageBlock + j * kThreads + threadIdx.x;
    upto += q <= M && live_page(C, q) ? 1 : 0;
  }
  upto = block_sum(upto);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    w.total[0] = M;
    w.total[1] = M - upto;  // pages that move
    if (num_live) *num_live = M;
  }
  const int p0 = blockIdx.x * kPageBlock + threadIdx.x * kPer;
  uint32_t mask = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) mask |= (live_page(C, p0 + j) ? 1u : 0u) << j;
  int total;
  int lives = before + block_scan(__popc(mask), total);  // live pages before this one
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int q = p0 + j;
    if (q >= C.num_pages) break;
    const bool live = mask >> j & 1;
    w.list_b[q] = live && q > M ? lives - upto : -1;
    if (live && q > M) w.list_a[lives - upto] = q;
    if (!live && q > 0 && q <= M) w.list_a[C.num_pages / 2 + (q - 1 - lives)] = q;
    lives += live ? 1 : 0;
  }
}

constexpr int kCopyVecs = 4;  // 16-byte vectors in flight per thread

// Copies n 16-byte vectors by the whole block, kCopyVecs loads in flight per thread.
__device__ __forceinline__ void copy_vecs(uint4* d, const uint4* s, int64_t first, int64_t n) {
  for (int64_t j = first + threadIdx.x; j < n; j += kThreads * kCopyVecs) {
    uint4 v[kCopyVecs];
#pragma unroll
    for (int u = 0; u < kCopyVecs; ++u)
      if (j + u * kThreads < n) v[u] = s[j + u * kThreads];
#pragma unroll
    for (int u = 0; u < kCopyVecs; ++u)
      if (j + u * kThreads < n) d[j + u * kThreads] = v[u];
  }
}

// Blocks walk over (mover, K or V, 16 KiB piece) units, then over the block table: HBM bounds it (with 137
// MB of pages to move 39 us = 7 TB/s of reads and writes; 58 us for the call, which counts and plans before).
__global__ void __launch_bounds__(kThreads) move_kernel(PageRowsLaunch p) {
  const KvDev& C = p.cache;
  const Ws w = carve(p.ws, C.num_pages, 0);
  let_next();
  wait_prior();
  const int moved = w.total[1];
  const int32_t* holes = w.list_a + C.num_pages / 2;
  const int64_t vecs = (int64_t)C.Hkv * C.page_size * C.d * p.es / 16;
  const int pieces = (int)((vecs + 1023) / 1024);
  const int64_t units = (int64_t)moved * 2 * pieces;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int piece = (int)(u % pieces);
    const int64_t item = u / pieces;
    const int src = w.list_a[item >> 1], dst = holes[item >> 1];
    uint8_t* pool = static_cast<uint8_t*>((item & 1) ? C.v : C.k);
    copy_vecs(reinterpret_cast<uint4*>(pool + (int64_t)dst * C.page_stride * p.es),
              reinterpret_cast<const uint4*>(pool + (int64_t)src * C.page_stride * p.es), (int64_t)piece * 1024,
              min(vecs, (int64_t)(piece + 1) * 1024));
  }
  const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
  for (int64_t r = at; r < moved; r += step) {
    const int src = w.list_a[r], dst = holes[r];
    C.refcount[dst] = C.refcount[src];
    C.refcount[src] = 0;
  }
  const int64_t entries = (int64_t)C.num_table_rows * C.max_pages;
  for (int64_t e = at; e < entries; e += step) {
    const int id = C.table[e];
    if (id <= 0) continue;
    if (id >= C.num_pages) {
      set_status(p.status, GDN_STATUS_PAGE_RANGE);
      continue;
    }
    const int r = w.list_b[id];
    if (r >= 0) C.table[e] = holes[r];
  }
}

// ---- copies of whole items ------------------------------------------------------------------------

__global__ void __launch_bounds__(kThreads) copy_items_kernel(CopyLaunch p, int pieces0, int pieces) {
  let_next();
  wait_prior();
  const int64_t units = (int64_t)p.count * pieces;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = (int)(u / pieces);
    int piece = (int)(u - (int64_t)i * pieces);
    const int src = load(p.src + i), dst = load(p.dst + i);
    if (src >= p.limit || dst >= p.limit) {
      if (threadIdx.x == 0) set_status(p.status, p.range_bit);
      continue;
    }
    if (dst <= 0 || (src <= 0 && !p.null_zeros) || src == dst) continue;
    const int j = piece >= pieces0 ? 1 : 0;
    if (j) piece -= pieces0;
    const int64_t n = p.bytes[j] / 16, first = (int64_t)piece * 1024, last = min(n, first + 1024);
    uint4* d = reinterpret_cast<uint4*>(p.pool[j] + (int64_t)dst * p.stride[j]);
    if (src <= 0) {
      for (int64_t q = first + threadIdx.x; q < last; q += kThreads) d[q] = make_uint4(0, 0, 0, 0);
    } else {
      copy_vecs(d, reinterpret_cast<const uint4*>(p.pool[j] + (int64_t)src * p.stride[j]), first, last);
    }
  }
}

// Launch as a programmatic dependent of the kernel just before it on the stream.
template <typename... P, typename... A>
cudaError_t launch_of(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, cudaStream_t s, A... args) {
  return launch_of(kernel, grid, kThreads, s, args...);
}
cudaError_t launch_hand_out(void (*kernel)(PageRowsLaunch), cudaStream_t s, const PageRowsLaunch& p) {
  return launch_of(kernel, dim3(kHandCtas), kHandThreads, s, p);
}

constexpr int kCopyBlocks = kSms * 8;  // two thousand threads per SM

}  // namespace

size_t kv_workspace_ints(int32_t num_pages, int32_t count) {
  return (size_t)5 * count + max_of(page_blocks(num_pages), 8) + 4 + 2 * (size_t)num_pages;
}

cudaError_t launch_kv_append(const AppendLaunch& p, cudaStream_t s) {
  return launch_after(append_kernel, dim3((p.rows.num_tokens + kThreads / 32 - 1) / (kThreads / 32)), s, p);
}

cudaError_t launch_kv_reserve(const PageRowsLaunch& p, cudaStream_t s) {
  const int nb = page_blocks(p.cache.num_pages);
  if (p.cache.num_pages <= kHandPages) return launch_hand_out(hand_out_kernel<false>, s, p);
  cudaError_t e = launch_after(need_kernel<false>, dim3(nb + p.count), s, p);
  if (e == cudaSuccess) e = launch_after(free_list_kernel, dim3(nb + 1), s, p);
  if (e == cudaSuccess) e = launch_after(reserve_kernel, dim3(p.count), s, p);
  return e;
}

cudaError_t launch_kv_release(const PageRowsLaunch& p, cudaStream_t s) {
  const int per_row = (p.cache.max_pages + kThreads - 1) / kThreads;
  return launch_after(release_kernel, dim3(per_row < 64 ? per_row : 64, p.count < 65535 ? p.count : 65535), s, p);
}

cudaError_t launch_kv_fork(const PageRowsLaunch& p, cudaStream_t s) {
  const int nb = page_blocks(p.cache.num_pages);
  cudaError_t e;
  if (p.cache.num_pages <= kHandPages && p.cache.max_pages <= kHandEntries) {
    e = launch_hand_out(hand_out_kernel<true>, s, p);
  } else {
    e = launch_after(need_kernel<true>, dim3(nb + p.count), s, p);
    if (e == cudaSuccess) e = launch_after(free_list_kernel, dim3(nb + 1), s, p);
    if (e == cudaSuccess) e = launch_after(fork_kernel, dim3(p.count), s, p);
  }
  if (e == cudaSuccess) e = launch_after(fork_copy_kernel, dim3(p.count, p.cache.Hkv, 2), s, p);
  return e;
}

cudaError_t launch_kv_compact(const PageRowsLaunch& p, int32_t* num_live, cudaStream_t s) {
  const int nb = page_blocks(p.cache.num_pages);
  cudaError_t e = launch_after(live_kernel, dim3(nb), s, p);
  if (e == cudaSuccess) e = launch_after(plan_kernel, dim3(nb), s, p, num_live);
  if (e == cudaSuccess) e = launch_after(move_kernel, dim3(kCopyBlocks), s, p);
  return e;
}

cudaError_t launch_copy_items(const CopyLaunch& p, cudaStream_t s) {
  const int pieces0 = (int)((p.bytes[0] / 16 + 1023) / 1024);
  const int pieces = pieces0 + (int)((p.bytes[1] / 16 + 1023) / 1024);
  const int64_t units = (int64_t)p.count * pieces;
  return launch_after(copy_items_kernel, dim3((int)(units < kCopyBlocks ? units : kCopyBlocks)), s, p, pieces0, pieces);
}

}  // namespace gdn
