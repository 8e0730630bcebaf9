// gdn_attn_plan.cuh -- the plan of attention over groups: the parts of groups and of rows, and the places of tokens.
//
// Group g shares min(prefix_lens[g], tokens before the new ones of its rows), down to whole pages, where two of its rows or
// more have new tokens that are well formed; what a row has of its own begins there.
#pragma once

#include "gdn_kv.cuh"

namespace gdn {

// The group's rows [a, b); false (and the status bit) for bounds that are none.  (Where all groups' are some, no row is in two.)
__device__ __forceinline__ bool group_bounds(int a, int b, int num_seqs, uint32_t* st) {
  if (a >= 0 && b >= a && b <= num_seqs) return true;
  set_status(st, GDN_STATUS_ROW_RANGE);
  return false;
}

// Whether row n's local tokens are some of the call's.  (Where all rows' are, rows follow one another and no token is in two.  With
// one that is not, a token may be in several rows, or between a group's first and last without being of its rows: nothing is
// shared then, and every row that is well formed goes over its own cache.)
__device__ __forceinline__ bool row_bounds(const KvRowsDev& R, int n) {
  const int a = load(R.qsl + n), b = load(R.qsl + n + 1);
  return a >= 0 && b >= a && b <= R.num_tokens;
}

// What a group's rows say together: those with new tokens that are well formed.
struct GroupRows {
  int count;
  int first;           // the first of them
  int least;           // tokens before the new ones, of the row that has fewest
  int bos, eos;        // their local tokens
  int pos_max;         // the highest position of a query (the lowest is `least`)
  __device__ GroupRows() : count(0), first(INT32_MAX), least(INT32_MAX), bos(INT32_MAX), eos(0), pos_max(0) {}
  __device__ __forceinline__ void add(int n, int row_bos, int len, int kv) {
    ++count;
    first = min(first, n);
    least = min(least, kv - len);
    bos = min(bos, row_bos);
    eos = max(eos, row_bos + len);
    pos_max = max(pos_max, kv - 1);
  }
  __device__ __forceinline__ void warp_meet() {
    count = __reduce_add_sync(0xffffffffu, count);
    first = __reduce_min_sync(0xffffffffu, first);
    least = __reduce_min_sync(0xffffffffu, least);
    bos = __reduce_min_sync(0xffffffffu, bos);
    eos = __reduce_max_sync(0xffffffffu, eos);
    pos_max = __reduce_max_sync(0xffffffffu, pos_max);
  }
  // Tokens that the group shares, of `prefix` given ones; seen: some query sees some of them.  (Behind all windows, with
  // nothing in front that stays visible, none does.)
  __device__ __forceinline__ int shared(int prefix, int page_size, int window, int sinks, bool& seen) const {
    int n = count >= 2 ? min(max(prefix, 0), least) : 0;
    n &= -page_size;
    const int low = window > 0 ? max(0, least - window + 1) : 0;
    seen = n > low || (n > 0 && min(sinks, low) > 0);
    return n;
  }
  __device__ __forceinline__ PartRec record(int tokens, int trow) const {
    return {bos, eos - bos, 0, tokens, trow, least, pos_max, 0};
  }
};

// A plan of few rows is made by every CTA of the pass for itself, which saves the launch of a kernel for it.  (The join reads
// the first one's.)  scratch: kPlanInts, 16-byte aligned; returns the parts there.  All threads call.
constexpr int kPlanRows = 256, kPlanGroups = 32;
constexpr int kPlanRecs = (kPlanRows + kPlanGroups) * (int)(sizeof(PartRec) / 4);
constexpr int kPlanInts = kPlanRecs + 5 * kPlanRows + 2 * kPlanGroups + 1;

template <int THREADS>
__device__ const PartRec* plan_here(const AttnLaunch& p, int* scratch) {
  const PartDev& part = p.part;
  const KvRowsDev& R = p.rows;
  const int tid = threadIdx.x, lane = tid & 31;
  PartRec* near = reinterpret_cast<PartRec*>(scratch);
  int* first = scratch + kPlanRecs;    // of a row: query_start_loc
  int* len = first + kPlanRows;        // new tokens, 0 for a row that is none
  int* kv = len + kPlanRows;
  int* trow = kv + kPlanRows;
  int* own = trow + kPlanRows;         // first own token, + 1 where its group's shared ones are seen
  int* start = own + kPlanRows;        // of a group
  int* prefix = start + kPlanGroups + 1;
  uint32_t* st = blockIdx.x == 0 ? p.status : nullptr;
  // (groups' loads go out before rows' come back)
  static_assert(kPlanGroups < THREADS, "a thread per group");
  int g0 = 0, g1 = 0, given = 0;
  if (tid <= part.groups) g0 = load(part.start + tid);
  if (tid < part.groups) {
    g1 = load(part.start + tid + 1);
    given = load(part.prefix + tid);
  }
  bool ascend = true;
  for (int n = tid; n < R.num_seqs; n += THREADS) {
    KvRow r;
    ascend &= row_bounds(R, n);
    const bool there = load_kv_row(R, p.cache, n, r, st);
    first[n] = r.bos;
    len[n] = there ? r.len : 0;
    kv[n] = r.kv;
    trow[n] = r.trow;
    own[n] = 0;
  }
  if (tid <= part.groups) start[tid] = g0;
  if (tid < part.groups) prefix[tid] = given;
  ascend = __syncthreads_and(ascend);
  const bool none = __syncthreads_or(tid < part.groups && !group_bounds(g0, g1, R.num_seqs, st)) || !ascend;  // nothing is shared
  PartRec* recs = part_recs(part);
  int2* token = part_tokens(part);
  for (int g = tid >> 5; g < part.groups; g += THREADS / 32) {
    const int a = start[g], b = start[g + 1];
    GroupRows s;
    bool seen = false;
    int tokens = 0;
    if (!none) {
      for (int n = a + lane; n < b; n += 32)
        if (len[n] > 0) s.add(n, first[n], len[n], kv[n]);
      s.warp_meet();
      tokens = s.shared(prefix[g], p.cache.page_size, p.window, p.sinks, seen);
      for (int n = a + lane; n < b; n += 32) own[n] = tokens + (seen ? 1 : 0);
    }
    if (lane == 0) recs[g] = near[g] = seen ? s.record(tokens, trow[s.first]) : PartRec{};
  }
  __syncthreads();
  for (int n = tid; n < R.num_seqs; n += THREADS)
    recs[part.groups + n] = near[part.groups + n] =
        len[n] > 0 ? PartRec{first[n], len[n], own[n] & ~1, kv[n], trow[n], kv[n] - len[n], kv[n] - 1, 0} : PartRec{};
  // The pass itself looks tokens up under a window, in its CTA's copy; the join does in any case, in the first, which the
  // CTAs fill together where they need none of their own.
  const bool all = p.window > 0;
  if (!all) token = part.token;
  for (int i = all ? tid : tid * gridDim.x + blockIdx.x; i < R.num_tokens; i += all ? THREADS : THREADS * gridDim.x) {
    int n = 0;  // the last row that begins at or before the token, or, of bounds that do not ascend, the last one that holds it
    if (ascend) {
      for (int step = kPlanRows / 2; step; step >>= 1)
        if (n + step < R.num_seqs && first[n + step] <= i) n += step;
    } else {
      for (n = R.num_seqs - 1; n > 0 && !(i >= first[n] && i < first[n] + len[n]);) --n;
    }
    const bool there = i >= first[n] && i < first[n] + len[n];
    token[i] = there ? make_int2(kv[n] - len[n] + i - first[n], own[n] & 1) : make_int2(-1, 0);
  }
  __syncthreads();
  return near;
}

}  // namespace gdn
