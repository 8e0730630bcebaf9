// gdn_kv_groups.cu -- groups of rows that hold the same pages: how far they agree, and the plan of attention over them.
//
// Both read a few integers per row and entry, 4 bytes an entry and row: what takes time is the launch and the loads that
// depend on one another (bounds, rows, table).
#include <algorithm>

#include "gdn_attn_plan.cuh"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kCluster = 8;

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_rank() {
  int r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The value that CTA `rank` of the cluster holds at `mine` of its shared memory.
__device__ __forceinline__ int from_rank(const int* mine, int rank) {
  uint32_t a;
  int v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Sets `mine` of CTA `rank` of the cluster.
__device__ __forceinline__ void to_rank(int* mine, int rank, int v) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

__device__ __forceinline__ bool group_rows(const GroupsLaunch& p, int g, int& a, int& b, uint32_t* st) {
  a = load(p.start + g);
  b = load(p.start + g + 1);
  return group_bounds(a, b, p.rows.num_seqs, st);
}
__device__ __forceinline__ void add_row(const GroupsLaunch& p, int n, GroupRows& s, uint32_t* st) {
  KvRow r;
  if (load_kv_row(p.rows, p.cache, n, r, st) && r.len > 0) s.add(n, r.bos, r.len, r.kv);
}

// ---- common prefix ----------------------------------------------------------------------------

__device__ __forceinline__ int table_row_of(const GroupsLaunch& p, int n) {
  return p.rows.table_rows ? load(p.rows.table_rows + n) : n;
}
__device__ __forceinline__ const int32_t* entries_of(const GroupsLaunch& p, int n) {
  return p.cache.table + (int64_t)table_row_of(p, n) * p.cache.max_pages;
}

// A cluster per group, or `clusters` of them, which meet in prefix[g] (set to the highest value before).  Its warps take runs
// of kRun entries of the rows in turn, those of all rows' beginnings first, and compare them with those of the group's
// first row; what lies behind a place where rows were seen to part is left out.
// 16 groups of 9 to 24 rows that share up to 8192 entries: 59 us with a warp per row, 9.6 so; what bounds it is its chain of
// loads: bounds, rows, entries (5 MB in all; 4 rows of 777 tokens take 3.2).
constexpr int kAhead = 8;  // entries of a lane that are on their way
constexpr int kRun = 32 * kAhead;

__global__ void __launch_bounds__(kThreads) begin_kernel(GroupsLaunch p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int g = blockIdx.x * kThreads + threadIdx.x;
  if (g < p.num_groups) p.prefix[g] = INT32_MAX;
}

template <int THREADS>
__global__ void __cluster_dims__(kCluster) __launch_bounds__(THREADS) common_kernel(GroupsLaunch p, int clusters) {
  constexpr int kWarps = THREADS / 32;
  __shared__ int least[kWarps], first[kWarps];
  __shared__ int agree;
  const int cluster = blockIdx.x / kCluster, g = cluster / clusters, mine = cluster - g * clusters, rank = cluster_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int a, b;
  uint32_t* st = mine == 0 && rank == 0 ? p.status : nullptr;
  if (!group_rows(p, g, a, b, st)) a = b = 0;
  GroupRows s;
  for (int n = a + (int)threadIdx.x; n < b; n += THREADS) add_row(p, n, s, st);
  s.warp_meet();
  if (lane == 0) {
    least[warp] = s.least;
    first[warp] = s.first;
  }
  __syncthreads();
  s.least = __reduce_min_sync(0xffffffffu, lane < kWarps ? least[lane] : INT32_MAX);
  s.first = __reduce_min_sync(0xffffffffu, lane < kWarps ? first[lane] : INT32_MAX);
  const int whole = s.first != INT32_MAX ? s.least / p.cache.page_size : 0;
  if (threadIdx.x == 0) agree = whole;
  __syncthreads();
  if (whole > 0) {
    const int32_t* of_first = entries_of(p, s.first);
    const int rows = b - a;
    const int64_t runs = (int64_t)((whole + kRun - 1) / kRun) * rows;
    for (int64_t i = (mine * kCluster + rank) * kWarps + warp; i < runs; i += clusters * kCluster * kWarps) {
      const int n = a + (int)(i % rows), e0 = (int)(i / rows) * kRun;
      // (one lane reads it, as others' warps lower it and this one's first lane just did: all lanes stay or all leave)
      const int until = lane == 0 ? *(volatile int*)&agree : 0;
      if (e0 >= __shfl_sync(0xffffffffu, until, 0)) break;
      KvRow r;
      if (n == s.first || !load_kv_row(p.rows, p.cache, n, r, nullptr) || r.len == 0) continue;
      const int32_t* of_row = p.cache.table + (int64_t)r.trow * p.cache.max_pages;
      bool differs[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int e = e0 + 32 * u + lane;
        differs[u] = e < whole && page_or_null(load(of_first + e), p.cache, p.status) !=
                                      page_or_null(load(of_row + e), p.cache, p.status);
      }
      int at = whole;
#pragma unroll
      for (int u = kAhead - 1; u >= 0; --u) {
        const unsigned m = __ballot_sync(0xffffffffu, differs[u]);
        if (m) at = e0 + 32 * u + __ffs(m) - 1;
      }
      if (at < whole && lane == 0) atomicMin(&agree, at);
    }
  }
  __syncthreads();
  cluster_sync();
  if (rank == 0 && warp == 0) {
    int v = lane < kCluster ? from_rank(&agree, lane) : INT32_MAX;
    v = __reduce_min_sync(0xffffffffu, v);
    if (lane == 0 && clusters == 1) p.prefix[g] = v * p.cache.page_size;
    if (lane == 0 && clusters > 1) atomicMin(p.prefix + g, v * p.cache.page_size);
  }
  cluster_sync();  // (no CTA ends while another reads its shared memory)
}

// ---- the plan ---------------------------------------------------------------------------------

// A row's new tokens, each with its position: a lane per row takes them one by one, which does for verify rows; the
// caller's lanes take long rows' together.
__device__ __forceinline__ void place_tokens(int2* token, const KvRow& r, int from, int step, int shares) {
  for (int t = from; t < r.len; t += step) token[r.bos + t] = make_int2(r.kv - r.len + t, shares);
}

// One cluster: the parts of rows, a thread (or, where rows may be long, a warp) each, then those of groups, a warp each, which
// move the beginnings of their rows' own parts.
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads) group_plan_kernel(GroupsLaunch p) {
  constexpr int kAll = kCluster * kThreads;
  __shared__ int none;  // nothing is shared
  const int lane = threadIdx.x & 31;
  const int me = blockIdx.x * kThreads + threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = me; i < p.rows.num_tokens; i += kAll) p.token[i] = make_int2(-1, 0);
  if (threadIdx.x == 0) none = 0;
  cluster_sync();
  const bool lanes = p.rows.max_q > 64;  // a row's tokens go to a warp's lanes
  bool bad = false;  // bounds of a row or a group
  for (int n = lanes ? me >> 5 : me; n < p.rows.num_seqs; n += lanes ? kAll / 32 : kAll) {
    KvRow r;
    PartRec rec{};
    bad |= !row_bounds(p.rows, n);
    if (load_kv_row(p.rows, p.cache, n, r, p.status) && r.len > 0) {
      rec = {r.bos, r.len, 0, r.kv, r.trow, r.kv - r.len, r.kv - 1, 0};
      place_tokens(p.token, r, lanes ? lane : 0, lanes ? 32 : 1, 0);
    }
    if (!lanes || lane == 0) p.recs[p.num_groups + n] = rec;
  }
  for (int g = me; g < p.num_groups; g += kAll) {
    int a, b;
    bad |= !group_rows(p, g, a, b, p.status);
  }
  for (int rank = 0; bad && rank < kCluster; ++rank) to_rank(&none, rank, 1);
  cluster_sync();
  for (int g = me >> 5; g < p.num_groups; g += kAll / 32) {
    int a, b;
    if (none || !group_rows(p, g, a, b, nullptr)) a = b = 0;
    GroupRows s;
    for (int n = a + lane; n < b; n += 32) add_row(p, n, s, nullptr);
    s.warp_meet();
    bool seen;
    const int shared = s.shared(load(p.prefix + g), p.cache.page_size, p.window, p.sinks, seen);
    for (int i = a; shared > 0 && i < b; i += lanes ? 1 : 32) {
      const int n = lanes ? i : i + lane;
      KvRow r;
      if (n >= b || !load_kv_row(p.rows, p.cache, n, r, nullptr) || r.len == 0) continue;
      if (!lanes || lane == 0) p.recs[p.num_groups + n].from = shared;
      if (seen) place_tokens(p.token, r, lanes ? lane : 0, lanes ? 32 : 1, 1);
    }
    if (lane == 0) {
      const PartRec rec = seen ? s.record(shared, table_row_of(p, s.first)) : PartRec{};
      p.recs[g] = rec;
    }
  }
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), int blocks, int threads, cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

// Blocks of 1024 threads where a group's rows may have more entries than a cluster of smaller ones takes at once: those 16
// groups 11 us, with blocks of 256 19; 4 rows of 64 entries 3.6 us with blocks of 1024, 3.2 with 256.  And as many clusters
// a group as have 65536 entries each to go over at once, behind a launch that sets what they meet in: one group of 16 rows of
// 8192 entries 5.7 us instead of 6.8, of 64 6 (18), of 256 7.5 (60); those 16 groups 9.6.
cudaError_t launch_kv_common_prefix(const GroupsLaunch& p, cudaStream_t s) {
  const int64_t entries = (int64_t)p.cache.max_pages * p.rows.num_seqs / p.num_groups;
  if (entries <= kCluster * kThreads * kAhead)
    return launch(common_kernel<kThreads>, p.num_groups * kCluster, kThreads, s, p, 1);
  const int clusters = (int)std::min<int64_t>(entries / (kCluster * 1024 * kAhead), 2 * kSms / kCluster / p.num_groups);
  if (clusters < 2) return launch(common_kernel<1024>, p.num_groups * kCluster, 1024, s, p, 1);
  const cudaError_t e = launch(begin_kernel, (p.num_groups + kThreads - 1) / kThreads, kThreads, s, p);
  return e != cudaSuccess ? e : launch(common_kernel<1024>, p.num_groups * clusters * kCluster, 1024, s, p, clusters);
}

// Every CTA goes over all rows, groups and tokens then, a warp per group.  Against a kernel for the plan, us a call behind 777 shared
// tokens, 20 own ones each (d = 128, 16/2 heads): 4 rows of a group 12.3 (14.5), 256 rows 33 (38); d = 64, 8/2 heads: 16 groups
// of 16 rows of 4 tokens 35 (37), 32 of 8 38 (40); 64 of 4 were even.  In the pass on the CUDA cores, whose CTAs have 4 warps for
// 12 (of 8), behind a shorter prefix 1 x 64 x 4 17 (20), 16 x 16 x 4 32 (33), 32 x 8 x 4 35 (33), 64 x 4 x 4 40 (33).
bool group_plan_here(const AttnLaunch& p) {
  return p.rows.num_seqs <= kPlanRows && p.part.groups <= (p.part.quads ? kPlanGroups : kPlanGroups / 2) &&
         p.rows.num_tokens <= 4 * kPlanRows;
}

cudaError_t launch_group_plan(const GroupsLaunch& p, cudaStream_t s) {
  return launch(group_plan_kernel, kCluster, kThreads, s, p);
}

}  // namespace gdn
