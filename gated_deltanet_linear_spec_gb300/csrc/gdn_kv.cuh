// gdn_kv.cuh -- device-side types of the paged key-value cache and its launchers (not part of the ABI).
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

constexpr int kSms = 152;

// The cache as the kernels see it (plain values copied from gdn_kv_cache).
struct KvDev {
  void* k;
  void* v;
  int64_t page_stride;  // elements
  int32_t* table;
  int32_t* refcount;
  int32_t num_pages, num_table_rows, max_pages, page_size, Hkv, d;
};

// One subset of rows (plain values copied from gdn_kv_rows).
struct KvRowsDev {
  const int32_t* qsl;
  const int32_t* tok;         // NULL = identity
  const int32_t* table_rows;  // NULL = identity
  const int32_t* kv_lens;
  int32_t num_seqs, num_tokens, max_q;
};

// What the calls read, by coherent loads: a kernel here starts while the one before it still runs, so lines of the
// table, the pages and the rows may change between its start and its griddepcontrol.wait, which rules out the
// read-only path (ld.global.nc, __ldg).
template <typename T>
__device__ __forceinline__ T load(const T* p) {
  __builtin_assume(__isGlobal(p));  // (else a generic load, which waits for stores to shared memory)
  return *p;
}

struct KvRow {
  int32_t bos, len;  // local tokens
  int32_t kv;        // cache length with them
  int32_t trow;      // row of the block table
};

// A row's values, checked against the tensors they index; false (and the status bit) for a bad one.
__device__ __forceinline__ bool check_kv_row(const KvRowsDev& R, const KvDev& C, int bos, int eos, int kv, int trow,
                                             KvRow& r, uint32_t* st) {
  r.bos = bos;
  r.kv = kv;
  r.trow = trow;
  r.len = 0;
  if (bos < 0 || eos < bos || eos > R.num_tokens || eos - bos > R.max_q || kv < eos - bos ||
      (int64_t)kv > (int64_t)C.max_pages * C.page_size) {
    set_status(st, GDN_STATUS_ROW_RANGE);
    return false;
  }
  if (trow < 0 || trow >= C.num_table_rows) {
    set_status(st, GDN_STATUS_PAGE_RANGE);
    return false;
  }
  r.len = eos - bos;
  return true;
}
__device__ __forceinline__ bool load_kv_row(const KvRowsDev& R, const KvDev& C, int n, KvRow& r, uint32_t* st) {
  return check_kv_row(R, C, load(R.qsl + n), load(R.qsl + n + 1), load(R.kv_lens + n),
                      R.table_rows ? load(R.table_rows + n) : n, r, st);
}

// A row that holds a local token, for one that a search among ascending bounds did not find: the bounds of a bad row may have
// stood in its way.  -1 for none, at once for tokens behind the last row.  All lanes of a warp call together.
__device__ __forceinline__ int row_past_bad_bounds(const KvRowsDev& R, int local) {
  const int lane = threadIdx.x & 31, end = load(R.qsl + R.num_seqs);
  if (end >= 0 && end <= local) return -1;
  for (int n0 = 0; n0 < R.num_seqs; n0 += 32) {
    const int n = n0 + lane;
    bool holds = false;
    if (n < R.num_seqs) {
      const int a = load(R.qsl + n), b = load(R.qsl + n + 1);
      holds = a >= 0 && a <= local && local < b && b <= R.num_tokens && b - a <= R.max_q;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, holds);
    if (m) return n0 + __ffs(m) - 1;
  }
  return -1;
}
// The row of a local token, which a search among ascending bounds found to be row n; false for a token of no good row.
__device__ __forceinline__ bool load_row_of_token(const KvRowsDev& R, const KvDev& C, int local, int n, KvRow& r, uint32_t* st) {
  const auto of_row = [&](int i) { return load_kv_row(R, C, i, r, st) && local >= r.bos && local < r.bos + r.len; };
  if (of_row(n)) return true;
  n = row_past_bad_bounds(R, local);
  return n >= 0 && of_row(n);
}

// Global token of local token i (identity when there is no token_indx), or -1 if out of range.
__device__ __forceinline__ int32_t kv_token(const KvRowsDev& R, int32_t i, int32_t num_global, uint32_t* st) {
  const int32_t g = R.tok ? load(R.tok + i) : i;
  if (g >= 0 && g < num_global) return g;
  set_status(st, GDN_STATUS_TOKEN_RANGE);
  return -1;
}

// A table entry as a page to read: its id, or 0 (no tokens) for NULL and out-of-range entries.
__device__ __forceinline__ int32_t page_or_null(int32_t id, const KvDev& C, uint32_t* st) {
  if (id >= C.num_pages) {
    set_status(st, GDN_STATUS_PAGE_RANGE);
    return 0;
  }
  return id > 0 ? id : 0;
}

struct AppendLaunch {
  KvDev cache;
  KvRowsDev rows;
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;  // elements
  int32_t num_global;
  int32_t es;  // bytes of an element
  uint32_t* status;
};

// One entry of a pass over parts of the rows' caches: what a group's queries share, or what a row has of its own.  Written on
// the device, groups first.
struct PartRec {
  int32_t bos, len;    // local tokens, whose queries of a kv-head go together; len 0: nothing to do
  int32_t from, end;   // cached tokens; from is a multiple of the page size
  int32_t trow;        // row of the block table
  int32_t lo, hi;      // lowest and highest position of a query
  int32_t pad;
};

// Where the pieces of a query's result over one part are: of the workers c0 to c1, the qi-th query of their unit; c0 < 0: one
// piece, in the query's own place.
struct PieceRange {
  int32_t c0, c1, qi, pad;
};

// n / by for 0 <= n < 2^31.  (A division by a value that only the call knows takes 100 cycles and more, and the beginnings and
// ends of a pass's units are full of them.  magic is off by less than 1, so the product is by less than n 2^-63 < 1 / by.)
inline uint64_t magic_of(int by) { return (1ull << 63) / by + 1; }
__device__ __forceinline__ int by_magic(int n, uint64_t magic) { return (int)__umul64hi((uint64_t)n << 1, magic); }

// A pass over parts, and where it leaves (m, l, o) of its pieces.  Queries are numbered (local token, q-head), those of groups'
// parts first, then those of rows' own.
struct PartDev {
  PartRec* recs;        // [count], those of groups first
  int32_t count;
  int32_t groups;       // of them, those of groups
  int32_t tokens;       // local tokens of the call
  int2* token;          // [tokens]: position (-1: of no well-formed row), whether its row shares a prefix
  const int32_t* start;   // [groups + 1] first rows of groups
  const int32_t* prefix;  // [groups] tokens that they may share
  int32_t plan_here;    // the pass makes recs and token itself, a copy of them for each CTA
  PieceRange* range;    // [2][tokens][Hq]
  float* ml;            // [2][tokens][Hq][2]: m (of the scores before their scale), l of a query in one piece
  float* o;             // [2][tokens][Hq][d], or with `quads` [d / 4][2][tokens][Hq][4]
  uint64_t g_magic, h_magic;  // magic_of q-heads per kv-head and kv-heads
  int32_t quads;        // o, here and in pieces, by four columns: what neighbouring queries write is side by side
};

// The plan as this CTA of a pass sees it.  (Where all CTAs write one copy, their stores to one place queue up: 4 us.)
__device__ __forceinline__ PartRec* part_recs(const PartDev& p) {
  return p.recs + (p.plan_here ? (size_t)blockIdx.x * p.count : 0);
}
__device__ __forceinline__ int2* part_tokens(const PartDev& p) {
  return p.token + (p.plan_here ? (size_t)blockIdx.x * p.tokens : 0);
}

struct AttnLaunch {
  KvDev cache;
  KvRowsDev rows;
  const void* q;
  void* out;
  int64_t q_stride, out_stride;  // elements
  int32_t num_global;
  int32_t Hq, G;
  float scale;
  int32_t window;  // 0 = none
  int32_t sinks;
  int32_t few;     // > 0: rows of up to so many queries per kv-head are the split kernel's, others the prompt one's
  void* ws;
  uint32_t* status;
  PartDev part;    // of passes over parts
};

// Heads turned by their tokens' positions, alone or on their way into the cache.
struct TurnLaunch {
  const uint64_t* turns;  // [rotary / 2]
  int32_t rotary, layout;
  float magnitude;
  int32_t d, Hq, num_tokens;
  const int32_t* positions;  // alone: [num_tokens]
  const void* q;
  void* q_out;
  int64_t q_stride, q_out_stride;  // elements
  // into the cache
  KvDev cache;
  KvRowsDev rows;
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;
  int32_t num_global;
  uint32_t* status;
};

// Groups of rows: group g is rows [start[g], start[g + 1]).
struct GroupsLaunch {
  KvDev cache;
  KvRowsDev rows;
  const int32_t* start;
  int32_t* prefix;  // [num_groups] shared tokens, read or written
  int32_t num_groups;
  int32_t window, sinks;
  PartRec* recs;    // the plan's: [num_groups + num_seqs]
  int2* token;      // [num_tokens]
  uint32_t* status;
};

// A list of table rows whose pages change.
struct PageRowsLaunch {
  KvDev cache;
  int32_t es;
  int32_t count;
  const int32_t* rows;      // reserve, release: table rows (NULL = identity); fork: destination rows
  const int32_t* src_rows;  // fork
  const int32_t* a;         // reserve: from_lens; release: first_page (NULL = 0); fork: lens
  const int32_t* b;         // reserve: to_lens; release: last_page (NULL = max_pages)
  int32_t* ws;
  uint32_t* status;
};

// Two pools copied item by item: item i moves `bytes[j]` bytes of pool j from src[i] to dst[i].
struct CopyLaunch {
  uint8_t* pool[2];
  int64_t stride[2];  // bytes from one item to the next
  int64_t bytes[2];   // multiples of 16
  const int32_t* src;
  const int32_t* dst;
  int32_t count;
  int32_t limit;      // ids are below this
  uint32_t range_bit;
  int32_t null_zeros;  // a NULL source: 1 = zeros, 0 = the pair is skipped
  uint32_t* status;
};

// Validation shared with the GDN entry points (gdn_abi.cu).
int check_layer_pools(const gdn_layer_desc* layer, const gdn_pools* pools);

// Ints of workspace that the page calls take (see gdn_kv_pages.cu for the layout).
size_t kv_workspace_ints(int32_t num_pages, int32_t count);

cudaError_t launch_kv_append(const AppendLaunch& p, cudaStream_t s);
cudaError_t launch_rope(const TurnLaunch& p, gdn_dtype dtype, cudaStream_t s);
cudaError_t launch_kv_append_rope(const TurnLaunch& p, gdn_dtype dtype, cudaStream_t s);
cudaError_t launch_kv_reserve(const PageRowsLaunch& p, cudaStream_t s);
cudaError_t launch_kv_release(const PageRowsLaunch& p, cudaStream_t s);
cudaError_t launch_kv_fork(const PageRowsLaunch& p, cudaStream_t s);
cudaError_t launch_kv_compact(const PageRowsLaunch& p, int32_t* num_live, cudaStream_t s);
cudaError_t launch_copy_items(const CopyLaunch& p, cudaStream_t s);

// Rows of up to 64 queries per kv-head (bf16, d = 64, 128, 256): split over the cache's length.
bool attn_split_supported(const AttnLaunch& p, gdn_dtype dtype);
size_t attn_split_workspace(const AttnLaunch& p);
cudaError_t launch_attn_split(const AttnLaunch& p, cudaStream_t s);
// Longer bf16 rows (d = 64, 128, 256): prompts, on tcgen05.
// What `few` of a call with both kinds of rows is; 0: all rows go one way.
int32_t attn_few(const AttnLaunch& p, gdn_dtype dtype);
bool attn_prompt_supported(const AttnLaunch& p, gdn_dtype dtype);
size_t attn_prompt_workspace(const AttnLaunch& p);
cudaError_t launch_attn_prompt(const AttnLaunch& p, cudaStream_t s);
// Every other layout, rows of any length: split over the cache's length, on the CUDA cores.
size_t attn_split_fma_workspace(const AttnLaunch& p);
cudaError_t launch_attn_split_fma(const AttnLaunch& p, gdn_dtype dtype, cudaStream_t s);

// Groups of rows over shared prefixes: the plan of their parts, passes over parts, and the join of what those leave.
cudaError_t launch_kv_common_prefix(const GroupsLaunch& p, cudaStream_t s);
bool group_plan_here(const AttnLaunch& p);  // the pass makes its plan itself
constexpr int kMaxPassCtas = 3 * kSms;      // of a pass over parts
cudaError_t launch_group_plan(const GroupsLaunch& p, cudaStream_t s);
// Where a pass leaves its pieces: [2 * workers][queries of a unit] (m, l), and o, with `quads` [2 * workers][d / 4][queries][4].
struct PartPieces {
  float* stats;
  float* o;
  int32_t queries;
  int32_t workers;
};
bool attn_shared_supported(const AttnLaunch& p, gdn_dtype dtype);  // on tcgen05: rows of up to a CTA's queries
size_t attn_shared_workspace(const AttnLaunch& p);
PartPieces attn_shared_pieces(const AttnLaunch& p, void* ws);
cudaError_t launch_attn_shared(const AttnLaunch& p, cudaStream_t s);
size_t attn_split_fma_parts_workspace(const AttnLaunch& p);
PartPieces attn_split_fma_parts_pieces(const AttnLaunch& p, void* ws);
cudaError_t launch_attn_split_fma_parts(const AttnLaunch& p, gdn_dtype dtype, cudaStream_t s);
cudaError_t launch_join_parts(const AttnLaunch& p, gdn_dtype dtype, PartPieces pieces, cudaStream_t s);

}  // namespace gdn
