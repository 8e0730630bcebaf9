// gdn_kv_abi.cu -- C entry points of the paged key-value cache: host-side validation and launches.
//
// As in gdn_abi.cu nothing here reads device memory, synchronises or allocates; what only device
// data can show is checked by the kernels and reported through the status word.
#include <limits.h>
#include <math.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include "gdn_kv.cuh"

using namespace gdn;

namespace {

constexpr int32_t kMaxTableEntries = 1 << 20;  // of one row: the sums of needs stay in 32 bits
constexpr int32_t kMaxPages = 1 << 28;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t round256(size_t b) { return (b + 255) & ~size_t(255); }
int es_of(gdn_dtype t) { return t == GDN_BF16 ? 2 : 4; }
int cuda_rc(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
};

// Sizes of a cache.
int check_shape(const gdn_kv_cache* c) {
  if (!c) return GDN_ERR_NULL_ARG;
  if (c->dtype != GDN_BF16 && c->dtype != GDN_F32) return GDN_ERR_DTYPE;
  if (c->num_pages < 2 || c->num_pages > kMaxPages) return GDN_ERR_SHAPE;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return GDN_ERR_SHAPE;
  if (c->num_kv_heads < 1 || c->num_kv_heads > 1024) return GDN_ERR_SHAPE;
  if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16) return GDN_ERR_SHAPE;
  const int64_t dense = (int64_t)c->num_kv_heads * c->page_size * c->head_dim;
  if (c->page_stride != 0 && (c->page_stride < dense || c->page_stride >= ((int64_t)1 << 38))) return GDN_ERR_SHAPE;
  if (c->page_stride * es_of(c->dtype) % 16) return GDN_ERR_ALIGN;
  // pages are whole slabs of page_size x head_dim apart, and slabs are numbered in 32 bits
  const int64_t slab = (int64_t)c->page_size * c->head_dim, stride = c->page_stride ? c->page_stride : dense;
  if (stride % slab || (c->num_pages - 1) * (stride / slab) + c->num_kv_heads > INT32_MAX) return GDN_ERR_SHAPE;
  return GDN_OK;
}

int check_table(const gdn_kv_cache* c) {
  if (!c->block_table) return GDN_ERR_NULL_ARG;
  if (c->num_table_rows < 1 || c->max_pages < 1 || c->max_pages > kMaxTableEntries) return GDN_ERR_SHAPE;
  if ((int64_t)c->max_pages * c->page_size > INT32_MAX) return GDN_ERR_SHAPE;
  return GDN_OK;
}

int check_pools(const gdn_kv_cache* c) {
  if (!c->k_pool || !c->v_pool) return GDN_ERR_NULL_ARG;
  return aligned16(c->k_pool) && aligned16(c->v_pool) ? GDN_OK : GDN_ERR_ALIGN;
}

int check_kv_rows(const gdn_kv_rows* r) {
  if (!r) return GDN_ERR_NULL_ARG;
  if (r->num_seqs < 0 || r->num_tokens < 0 || r->num_seqs > 65535) return GDN_ERR_SHAPE;
  if (r->num_seqs == 0) return r->num_tokens == 0 ? GDN_OK : GDN_ERR_SHAPE;
  if (!r->query_start_loc || !r->kv_lens) return GDN_ERR_NULL_ARG;
  return r->max_query_len >= 0 ? GDN_OK : GDN_ERR_SHAPE;
}

// A [tokens, heads, d] tensor: its stride in elements, 0 for a bad one.
int64_t token_stride(int64_t stride, int64_t dense, int es) {
  if (stride == 0) return dense;
  return stride >= dense && stride <= ((int64_t)1 << 40) && stride * es % 16 == 0 ? stride : 0;
}

int check_attn(const gdn_attn_desc* a, const gdn_kv_cache* c) {
  if (!a) return GDN_ERR_NULL_ARG;
  if (a->num_q_heads < 1 || a->num_q_heads > 65535 || a->num_q_heads % c->num_kv_heads) return GDN_ERR_SHAPE;
  if (a->num_sinks < 0) return GDN_ERR_SHAPE;
  return a->scale == a->scale && fabsf(a->scale) < INFINITY ? GDN_OK : GDN_ERR_SHAPE;
}

KvDev kv_dev(const gdn_kv_cache* c) {
  KvDev d{};
  d.k = c->k_pool;
  d.v = c->v_pool;
  d.page_stride = c->page_stride ? c->page_stride : (int64_t)c->num_kv_heads * c->page_size * c->head_dim;
  d.table = c->block_table;
  d.refcount = c->refcount;
  d.num_pages = c->num_pages;
  d.num_table_rows = c->num_table_rows;
  d.max_pages = c->max_pages;
  d.page_size = c->page_size;
  d.Hkv = c->num_kv_heads;
  d.d = c->head_dim;
  return d;
}

KvRowsDev kv_rows_dev(const gdn_kv_rows* r) {
  return KvRowsDev{r->query_start_loc, r->token_indx, r->table_rows, r->kv_lens,
                   r->num_seqs,        r->num_tokens, r->max_query_len};
}

AttnLaunch attn_args(const gdn_attn_desc* a, const gdn_kv_cache* c, const gdn_kv_rows* r) {
  AttnLaunch p{};
  p.cache = kv_dev(c);
  p.rows = kv_rows_dev(r);
  p.Hq = a->num_q_heads;
  p.G = a->num_q_heads / c->num_kv_heads;
  p.scale = a->scale > 0.f ? a->scale : 1.0f / sqrtf((float)c->head_dim);
  p.window = a->window > 0 ? a->window : 0;
  p.sinks = a->window > 0 ? a->num_sinks : 0;
  return p;
}

// What the calls that change pages share; `ws` says whether they need the workspace.
int page_call(const gdn_kv_cache* c, int32_t count, bool ws, void* workspace, size_t bytes) {
  int rc;
  if ((rc = check_shape(c)) || (rc = check_table(c))) return rc;
  if (!c->refcount) return GDN_ERR_NULL_ARG;
  if (count < 0) return GDN_ERR_SHAPE;
  if (!ws || count == 0) return GDN_OK;
  if (!workspace || bytes < gdn_kv_workspace_bytes(c, count)) return GDN_ERR_WORKSPACE;
  return (reinterpret_cast<uintptr_t>(workspace) & 255u) ? GDN_ERR_ALIGN : GDN_OK;
}

PageRowsLaunch page_args(const gdn_kv_cache* c, int32_t count, void* ws, uint32_t* status) {
  PageRowsLaunch p{};
  p.cache = kv_dev(c);
  p.es = es_of(c->dtype);
  p.count = count;
  p.ws = static_cast<int32_t*>(ws);
  p.status = status;
  return p;
}

}  // namespace

extern "C" {

size_t gdn_kv_workspace_bytes(const gdn_kv_cache* cache, int32_t count) {
  if (check_shape(cache) || count < 0) return 0;
  return round256(4 * kv_workspace_ints(cache->num_pages, count));
}

int gdn_kv_append(const gdn_kv_cache* cache, const gdn_kv_rows* rows, const void* k, int64_t k_stride, const void* v,
                  int64_t v_stride, int32_t num_global_tokens, uint32_t* d_status, void* stream) {
  Range range("gdn_kv_append");
  int rc;
  if ((rc = check_shape(cache)) || (rc = check_table(cache)) || (rc = check_pools(cache)) || (rc = check_kv_rows(rows)))
    return rc;
  if (num_global_tokens < 0) return GDN_ERR_SHAPE;
  if (rows->num_tokens == 0) return GDN_OK;
  if (!k || !v) return GDN_ERR_NULL_ARG;
  if (!aligned16(k) || !aligned16(v)) return GDN_ERR_ALIGN;
  if (!rows->token_indx && rows->num_tokens > num_global_tokens) return GDN_ERR_SHAPE;
  AppendLaunch p{};
  p.cache = kv_dev(cache);
  p.rows = kv_rows_dev(rows);
  p.es = es_of(cache->dtype);
  const int64_t dense = (int64_t)cache->num_kv_heads * cache->head_dim;
  p.k = k;
  p.v = v;
  p.k_stride = token_stride(k_stride, dense, p.es);
  p.v_stride = token_stride(v_stride, dense, p.es);
  if (!p.k_stride || !p.v_stride) return GDN_ERR_SHAPE;
  p.num_global = num_global_tokens;
  p.status = d_status;
  return cuda_rc(launch_kv_append(p, (cudaStream_t)stream));
}

size_t gdn_attention_workspace_bytes(const gdn_attn_desc* attn, const gdn_kv_cache* cache, const gdn_kv_rows* rows) {
  if (check_shape(cache) || check_table(cache) || check_attn(attn, cache) || check_kv_rows(rows)) return 0;
  if (rows->num_seqs == 0) return 0;
  AttnLaunch p = attn_args(attn, cache, rows);
  if (attn_split_supported(p, cache->dtype)) return round256(attn_split_workspace(p));
  if (!attn_prompt_supported(p, cache->dtype)) return round256(attn_split_fma_workspace(p));
  p.few = attn_few(p, cache->dtype);
  const size_t need = attn_prompt_workspace(p), split = p.few ? attn_split_workspace(p) : 0;
  return round256(need > split ? need : split);  // one after the other in one workspace
}

int gdn_paged_attention(const gdn_attn_desc* attn, const gdn_kv_cache* cache, const gdn_kv_rows* rows, const void* q,
                        int64_t q_stride, int32_t num_global_tokens, void* out, int64_t out_stride, void* workspace,
                        size_t workspace_bytes, uint32_t* d_status, void* stream) {
  Range range("gdn_paged_attention");
  int rc;
  if ((rc = check_shape(cache)) || (rc = check_table(cache)) || (rc = check_pools(cache)) ||
      (rc = check_attn(attn, cache)) || (rc = check_kv_rows(rows)))
    return rc;
  if (num_global_tokens < 0) return GDN_ERR_SHAPE;
  if (rows->num_tokens == 0) return GDN_OK;
  if (!q || !out) return GDN_ERR_NULL_ARG;
  if (!aligned16(q) || !aligned16(out)) return GDN_ERR_ALIGN;
  if (!rows->token_indx && rows->num_tokens > num_global_tokens) return GDN_ERR_SHAPE;
  if ((int64_t)rows->num_tokens * attn->num_q_heads > INT32_MAX) return GDN_ERR_SHAPE;
  const size_t need = gdn_attention_workspace_bytes(attn, cache, rows);
  if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 255u)) return GDN_ERR_ALIGN;
  AttnLaunch p = attn_args(attn, cache, rows);
  const int64_t dense = (int64_t)attn->num_q_heads * cache->head_dim;
  p.q = q;
  p.out = out;
  p.q_stride = token_stride(q_stride, dense, es_of(cache->dtype));
  p.out_stride = token_stride(out_stride, dense, es_of(cache->dtype));
  if (!p.q_stride || !p.out_stride) return GDN_ERR_SHAPE;
  p.num_global = num_global_tokens;
  p.ws = workspace;
  p.status = d_status;
  if (attn_split_supported(p, cache->dtype)) return cuda_rc(launch_attn_split(p, (cudaStream_t)stream));
  if (!attn_prompt_supported(p, cache->dtype))
    return cuda_rc(launch_attn_split_fma(p, cache->dtype, (cudaStream_t)stream));
  p.few = attn_few(p, cache->dtype);
  if (p.few && (rc = cuda_rc(launch_attn_split(p, (cudaStream_t)stream)))) return rc;
  return cuda_rc(launch_attn_prompt(p, (cudaStream_t)stream));
}

int gdn_kv_reserve(const gdn_kv_cache* cache, int32_t count, const int32_t* table_rows, const int32_t* from_lens,
                   const int32_t* to_lens, void* workspace, size_t workspace_bytes, uint32_t* d_status, void* stream) {
  Range range("gdn_kv_reserve");
  const int rc = page_call(cache, count, true, workspace, workspace_bytes);
  if (rc || count == 0) return rc;
  if (!from_lens || !to_lens) return GDN_ERR_NULL_ARG;
  PageRowsLaunch p = page_args(cache, count, workspace, d_status);
  p.rows = table_rows;
  p.a = from_lens;
  p.b = to_lens;
  return cuda_rc(launch_kv_reserve(p, (cudaStream_t)stream));
}

int gdn_kv_release(const gdn_kv_cache* cache, int32_t count, const int32_t* table_rows, const int32_t* first_page,
                   const int32_t* last_page, uint32_t* d_status, void* stream) {
  Range range("gdn_kv_release");
  const int rc = page_call(cache, count, false, nullptr, 0);
  if (rc || count == 0) return rc;
  PageRowsLaunch p = page_args(cache, count, nullptr, d_status);
  p.rows = table_rows;
  p.a = first_page;
  p.b = last_page;
  return cuda_rc(launch_kv_release(p, (cudaStream_t)stream));
}

int gdn_kv_fork(const gdn_kv_cache* cache, int32_t count, const int32_t* src_rows, const int32_t* dst_rows,
                const int32_t* lens, void* workspace, size_t workspace_bytes, uint32_t* d_status, void* stream) {
  Range range("gdn_kv_fork");
  int rc = page_call(cache, count, true, workspace, workspace_bytes);
  if (rc || (rc = check_pools(cache)) || count == 0) return rc;
  if (!src_rows || !dst_rows || !lens) return GDN_ERR_NULL_ARG;
  PageRowsLaunch p = page_args(cache, count, workspace, d_status);
  p.src_rows = src_rows;
  p.rows = dst_rows;
  p.a = lens;
  return cuda_rc(launch_kv_fork(p, (cudaStream_t)stream));
}

int gdn_kv_copy_pages(const gdn_kv_cache* cache, int32_t count, const int32_t* src_pages, const int32_t* dst_pages,
                      uint32_t* d_status, void* stream) {
  Range range("gdn_kv_copy_pages");
  int rc;
  if ((rc = check_shape(cache)) || (rc = check_pools(cache))) return rc;
  if (count < 0) return GDN_ERR_SHAPE;
  if (count == 0) return GDN_OK;
  if (!src_pages || !dst_pages) return GDN_ERR_NULL_ARG;
  const KvDev d = kv_dev(cache);
  const int es = es_of(cache->dtype);
  CopyLaunch p{};
  for (int j = 0; j < 2; ++j) {
    p.pool[j] = static_cast<uint8_t*>(j ? d.v : d.k);
    p.stride[j] = d.page_stride * es;
    p.bytes[j] = (int64_t)d.Hkv * d.page_size * d.d * es;
  }
  p.src = src_pages;
  p.dst = dst_pages;
  p.count = count;
  p.limit = d.num_pages;
  p.range_bit = GDN_STATUS_PAGE_RANGE;
  p.status = d_status;
  return cuda_rc(launch_copy_items(p, (cudaStream_t)stream));
}

int gdn_kv_compact(const gdn_kv_cache* cache, int32_t* num_live, void* workspace, size_t workspace_bytes,
                   uint32_t* d_status, void* stream) {
  Range range("gdn_kv_compact");
  int rc = page_call(cache, 0, false, nullptr, 0);
  if (rc || (rc = check_pools(cache))) return rc;
  if (!workspace || workspace_bytes < gdn_kv_workspace_bytes(cache, 0)) return GDN_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return GDN_ERR_ALIGN;
  const PageRowsLaunch p = page_args(cache, 0, workspace, d_status);
  return cuda_rc(launch_kv_compact(p, num_live, (cudaStream_t)stream));
}

int gdn_copy_slots(const gdn_layer_desc* layer, const gdn_pools* pools, int32_t count, const int32_t* src_slots,
                   const int32_t* dst_slots, uint32_t* d_status, void* stream) {
  Range range("gdn_copy_slots");
  const int rc = check_layer_pools(layer, pools);
  if (rc) return rc;
  if (count < 0 || pools->num_slots > INT32_MAX) return GDN_ERR_SHAPE;
  if (count == 0) return GDN_OK;
  if (!src_slots || !dst_slots) return GDN_ERR_NULL_ARG;
  CopyLaunch p{};
  const int64_t channels =
      2LL * layer->num_k_heads * layer->head_k_dim + (int64_t)layer->num_v_heads * layer->head_v_dim;
  p.pool[0] = reinterpret_cast<uint8_t*>(pools->ssm_pool);
  p.stride[0] = p.bytes[0] = (int64_t)layer->num_v_heads * layer->head_v_dim * layer->head_k_dim * 4;
  p.pool[1] = static_cast<uint8_t*>(pools->conv_pool);
  p.stride[1] = layer->conv_state_len * channels * es_of(layer->act_dtype);
  p.bytes[1] = pools->conv_pool ? p.stride[1] : 0;
  p.src = src_slots;
  p.dst = dst_slots;
  p.count = count;
  p.limit = (int32_t)pools->num_slots;
  p.range_bit = GDN_STATUS_SLOT_RANGE;
  p.null_zeros = 1;
  p.status = d_status;
  return cuda_rc(launch_copy_items(p, (cudaStream_t)stream));
}

}  // extern "C"
