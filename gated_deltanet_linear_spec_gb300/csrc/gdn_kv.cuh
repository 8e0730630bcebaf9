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

}  // namespace gdn
