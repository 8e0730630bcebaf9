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
constexpr int32_t kMaxPairs = 128;  // of a head

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

int check_rope(const gdn_rope_desc* r, int32_t head_dim) {
  if (!r || !r->turns) return GDN_ERR_NULL_ARG;
  if (r->rotary_dim < 2 || r->rotary_dim % 2 || r->rotary_dim > head_dim) return GDN_ERR_SHAPE;
  if (r->layout != GDN_ROPE_HALF && r->layout != GDN_ROPE_INTERLEAVED) return GDN_ERR_SHAPE;
  if (!(fabsf(r->magnitude) < INFINITY)) return GDN_ERR_SHAPE;
  return (reinterpret_cast<uintptr_t>(r->turns) & 7u) ? GDN_ERR_ALIGN : GDN_OK;
}

// Whether tokens written to `out` may be read from `x` by another thread, all of one type; strides and widths in elements.
// What a call writes has to be memory that it does not read (other columns of one wider tensor included) or, in place,
// what the same thread reads.
bool entangled(const void* x, int64_t x_stride, int64_t x_width, const void* out, int64_t out_stride, int64_t out_width,
               int64_t tokens, int es, bool in_place) {
  if (tokens < 1) return false;
  const int64_t a = (int64_t)reinterpret_cast<uintptr_t>(x), b = (int64_t)reinterpret_cast<uintptr_t>(out);
  const int64_t aw = x_width * es, bw = out_width * es, stride = x_stride * es;
  const __int128 steps = tokens - 1;  // (2^31 tokens of 2^42 bytes are more than 64 bits hold)
  const __int128 a_end = a + steps * stride + aw, b_end = b + steps * (out_stride * es) + bw;
  if (a_end <= b || b_end <= a || (in_place && a == b && (tokens == 1 || x_stride == out_stride))) return false;
  if (tokens == 1 || x_stride != out_stride) return true;
  const int64_t between = ((b - a) % stride + stride) % stride;
  return between < aw || stride - between < bw;
}

// A frequency as a 64-bit fraction of a turn; false for one that is none.
bool turn_fraction(double radians, uint64_t& fraction) {
  const double turns = radians / 6.283185307179586476925;
  if (!(fabs(turns) < 0x1p52)) return false;
  const double scaled = floor(ldexp(turns - floor(turns), 64) + 0.5);
  fraction = scaled < 0x1p64 ? (uint64_t)scaled : 0;  // (a whole turn)
  return true;
}

// The frequencies of gdn_rope_turns; false for values that make none.
bool rope_turns(const gdn_rope_freq& f, uint64_t* turns, float* magnitude) {
  const int r = f.rotary_dim;
  const bool scaled = f.scaling != GDN_ROPE_PLAIN;
  if (r < 2 || r > 2 * kMaxPairs || r % 2 || f.scaling < GDN_ROPE_PLAIN || f.scaling > GDN_ROPE_RAMP) return false;
  if (!(f.base > 1.0 && f.base < INFINITY) || (scaled && !(f.factor > 0.0 && f.factor < INFINITY))) return false;
  const bool parts = f.scaling == GDN_ROPE_BANDS || f.scaling == GDN_ROPE_RAMP;
  if (parts && !(f.original_len > 0.0 && f.original_len < INFINITY)) return false;
  const double low = f.low != 0.0 ? f.low : 1.0;
  const double high = f.high != 0.0 ? f.high : f.scaling == GDN_ROPE_RAMP ? 32.0 : 4.0;
  if (parts && !(low > 0.0 && low < high && high < INFINITY)) return false;
  const double two_pi = 6.283185307179586476925;
  const double base = f.scaling == GDN_ROPE_NTK && r > 2 ? f.base * pow(f.factor, (double)r / (r - 2)) : f.base;
  if (!(base > 0.0 && base < INFINITY)) return false;
  // the pair that turns so often over the original length
  auto pair_of = [&](double times) { return r * log(f.original_len / (two_pi * times)) / (2.0 * log(f.base)); };
  double from = 0.0, to = 0.0;
  if (f.scaling == GDN_ROPE_RAMP) {
    from = fmax(floor(pair_of(high)), 0.0);
    to = fmin(ceil(pair_of(low)), r - 1.0);
  }
  for (int i = 0; i < r / 2; ++i) {
    double w = pow(base, -2.0 * i / r);
    if (f.scaling == GDN_ROPE_LINEAR) w /= f.factor;
    if (parts) {
      const double keep = f.scaling == GDN_ROPE_BANDS ? (f.original_len * w / two_pi - low) / (high - low)
                                                      : 1.0 - (i - from) / fmax(to - from, 0.001);
      const double k = fmin(fmax(keep, 0.0), 1.0);
      w = k * w + (1.0 - k) * w / f.factor;
    }
    if (!turn_fraction(w, turns[i])) return false;
  }
  // (a context that is not stretched needs none)
  if (magnitude) *magnitude = f.scaling == GDN_ROPE_RAMP && f.factor > 1.0 ? (float)(0.1 * log(f.factor) + 1.0) : 1.f;
  return true;
}

void rope_args(const gdn_rope_desc* r, TurnLaunch& p) {
  p.turns = r->turns;
  p.rotary = r->rotary_dim;
  p.layout = r->layout;
  p.magnitude = r->magnitude == 0.f ? 1.f : r->magnitude;
}

int check_groups(const gdn_kv_groups* g) {
  if (!g) return GDN_ERR_NULL_ARG;
  if (g->num_groups < 0 || g->num_groups > 65535) return GDN_ERR_SHAPE;
  if (g->num_groups > 0 && (!g->group_start_loc || !g->prefix_lens)) return GDN_ERR_NULL_ARG;
  return GDN_OK;
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

// What the attention calls refuse before their workspace is looked at; GDN_OK with no tokens: there is nothing to do.
int attention_checks(const gdn_attn_desc* attn, const gdn_kv_cache* cache, const gdn_kv_rows* rows, const void* q,
                     int32_t num_global_tokens, const void* out) {
  int rc;
  if ((rc = check_shape(cache)) || (rc = check_table(cache)) || (rc = check_pools(cache)) ||
      (rc = check_attn(attn, cache)) || (rc = check_kv_rows(rows)))
    return rc;
  if (num_global_tokens < 0) return GDN_ERR_SHAPE;
  if (rows->num_tokens == 0) return GDN_OK;
  if (!q || !out) return GDN_ERR_NULL_ARG;
  if (!aligned16(q) || !aligned16(out)) return GDN_ERR_ALIGN;
  if (!rows->token_indx && rows->num_tokens > num_global_tokens) return GDN_ERR_SHAPE;
  return (int64_t)rows->num_tokens * attn->num_q_heads > INT32_MAX ? GDN_ERR_SHAPE : GDN_OK;
}

int attention_args(const gdn_attn_desc* attn, const gdn_kv_cache* cache, const gdn_kv_rows* rows, const void* q,
                   int64_t q_stride, int32_t num_global_tokens, void* out, int64_t out_stride, void* workspace,
                   size_t workspace_bytes, size_t need, uint32_t* d_status, AttnLaunch& p) {
  if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 255u)) return GDN_ERR_ALIGN;
  p = attn_args(attn, cache, rows);
  const int64_t dense = (int64_t)attn->num_q_heads * cache->head_dim;
  p.q = q;
  p.out = out;
  p.q_stride = token_stride(q_stride, dense, es_of(cache->dtype));
  p.out_stride = token_stride(out_stride, dense, es_of(cache->dtype));
  if (!p.q_stride || !p.out_stride) return GDN_ERR_SHAPE;
  p.num_global = num_global_tokens;
  p.ws = workspace;
  p.status = d_status;
  return GDN_OK;
}

int attend_whole(AttnLaunch& p, gdn_dtype dtype, cudaStream_t s) {
  if (attn_split_supported(p, dtype)) return cuda_rc(launch_attn_split(p, s));
  if (!attn_prompt_supported(p, dtype)) return cuda_rc(launch_attn_split_fma(p, dtype, s));
  p.few = attn_few(p, dtype);
  int rc;
  if (p.few && (rc = cuda_rc(launch_attn_split(p, s)))) return rc;
  return cuda_rc(launch_attn_prompt(p, s));
}

// The pass that goes over the parts of all groups and rows: tcgen05's, where the queries of a row fit a CTA (with few queries as
// with many: 4 rows of one group behind 65536 tokens, 16 q-heads, 2 kv-heads, d = 128, take 29 us, 61 on mma.sync with
// 16 queries a tile; 12 and 15 behind 777); the CUDA cores' for types that it does not take.  Longer rows on the tensor
// cores fill tiles of their own, and share nothing.
enum Pass { kNoPass, kTilePass, kFmaPass };
Pass pass_of(const AttnLaunch& p, int32_t num_groups, gdn_dtype dtype) {
  if (p.rows.num_tokens == 0 || num_groups == 0) return kNoPass;
  if (!attn_prompt_supported(p, dtype)) return kFmaPass;
  return attn_shared_supported(p, dtype) ? kTilePass : kNoPass;
}

// The workspace of attention over groups: the plan's parts and tokens, where queries' pieces are, results in one piece, and the
// pass's own.
struct SharedWs {
  size_t recs, token, range, ml, o, pass, end;
};
SharedWs shared_ws(const AttnLaunch& p) {
  SharedWs w{};
  const size_t tokens = p.rows.num_tokens, queries = 2 * tokens * p.Hq;
  w.recs = 0;
  const size_t copies = p.part.plan_here ? kMaxPassCtas : 1;
  w.token = round256(w.recs + copies * p.part.count * sizeof(PartRec));
  w.range = round256(w.token + copies * tokens * sizeof(int2));
  w.ml = round256(w.range + queries * sizeof(PieceRange));
  w.o = round256(w.ml + queries * 8);
  w.pass = round256(w.o + queries * p.cache.d * 4);
  w.end = w.pass + round256(p.part.quads ? attn_shared_workspace(p) : attn_split_fma_parts_workspace(p));
  return w;
}
// The parts of all groups and rows in one pass.
void all_parts(AttnLaunch& p, int32_t num_groups, Pass pass) {
  p.part.groups = num_groups;
  p.part.count = num_groups + p.rows.num_seqs;
  p.part.tokens = p.rows.num_tokens;
  p.part.g_magic = magic_of(p.G);
  p.part.h_magic = magic_of(p.cache.Hkv);
  p.part.quads = pass == kTilePass;
  p.part.plan_here = group_plan_here(p);
}

GroupsLaunch groups_args(const gdn_kv_cache* c, const gdn_kv_rows* r, const gdn_kv_groups* g, uint32_t* status) {
  GroupsLaunch p{};
  p.cache = kv_dev(c);
  p.rows = kv_rows_dev(r);
  p.start = g->group_start_loc;
  p.prefix = g->prefix_lens;
  p.num_groups = g->num_groups;
  p.status = status;
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

int gdn_rope_turns(const gdn_rope_freq* freq, uint64_t* turns, float* magnitude) {
  if (!freq || !turns) return GDN_ERR_NULL_ARG;
  return rope_turns(*freq, turns, magnitude) ? GDN_OK : GDN_ERR_SHAPE;
}

int gdn_rope_turns_of(const double* radians, int32_t count, uint64_t* turns) {
  if (!radians || !turns) return GDN_ERR_NULL_ARG;
  if (count < 1 || count > kMaxPairs) return GDN_ERR_SHAPE;
  for (int32_t i = 0; i < count; ++i)
    if (!turn_fraction(radians[i], turns[i])) return GDN_ERR_SHAPE;
  return GDN_OK;
}

int gdn_rope(const gdn_rope_desc* rope, int32_t num_heads, int32_t head_dim, gdn_dtype dtype, const int32_t* positions,
             int32_t num_tokens, const void* x, int64_t x_stride, void* out, int64_t out_stride, void* stream) {
  Range range("gdn_rope");
  if (dtype != GDN_BF16 && dtype != GDN_F32) return GDN_ERR_DTYPE;
  if (head_dim < 16 || head_dim > 256 || head_dim % 16 || num_heads < 1 || num_heads > 65535) return GDN_ERR_SHAPE;
  int rc = check_rope(rope, head_dim);
  if (rc) return rc;
  if (num_tokens < 0) return GDN_ERR_SHAPE;
  if (num_tokens == 0) return GDN_OK;
  if (!positions || !x || !out) return GDN_ERR_NULL_ARG;
  if (!aligned16(x) || !aligned16(out)) return GDN_ERR_ALIGN;
  TurnLaunch p{};
  rope_args(rope, p);
  const int64_t dense = (int64_t)num_heads * head_dim;
  const int es = es_of(dtype);
  p.q_stride = token_stride(x_stride, dense, es);
  p.q_out_stride = token_stride(out_stride, dense, es);
  if (!p.q_stride || !p.q_out_stride || entangled(x, p.q_stride, dense, out, p.q_out_stride, dense, num_tokens, es, true))
    return GDN_ERR_SHAPE;
  p.d = head_dim;
  p.Hq = num_heads;
  p.num_tokens = num_tokens;
  p.positions = positions;
  p.q = x;
  p.q_out = out;
  return cuda_rc(launch_rope(p, dtype, (cudaStream_t)stream));
}

int gdn_kv_append_rope(const gdn_kv_cache* cache, const gdn_kv_rows* rows, const gdn_rope_desc* rope, const void* k,
                       int64_t k_stride, const void* v, int64_t v_stride, int32_t num_q_heads, const void* q,
                       int64_t q_stride, void* q_out, int64_t q_out_stride, int32_t num_global_tokens, uint32_t* d_status,
                       void* stream) {
  Range range("gdn_kv_append_rope");
  int rc;
  if ((rc = check_shape(cache)) || (rc = check_table(cache)) || (rc = check_pools(cache)) ||
      (rc = check_kv_rows(rows)) || (rc = check_rope(rope, cache->head_dim)))
    return rc;
  if (num_global_tokens < 0 || num_q_heads < 0 || num_q_heads > 65535) return GDN_ERR_SHAPE;
  if (rows->num_tokens == 0) return GDN_OK;
  if (!k || !v || (num_q_heads > 0 && (!q || !q_out))) return GDN_ERR_NULL_ARG;
  if (!aligned16(k) || !aligned16(v)) return GDN_ERR_ALIGN;
  if (num_q_heads > 0 && (!aligned16(q) || !aligned16(q_out))) return GDN_ERR_ALIGN;
  if (!rows->token_indx && rows->num_tokens > num_global_tokens) return GDN_ERR_SHAPE;
  TurnLaunch p{};
  rope_args(rope, p);
  p.cache = kv_dev(cache);
  p.rows = kv_rows_dev(rows);
  const int es = es_of(cache->dtype);
  const int64_t dense = (int64_t)cache->num_kv_heads * cache->head_dim;
  p.k = k;
  p.v = v;
  p.k_stride = token_stride(k_stride, dense, es);
  p.v_stride = token_stride(v_stride, dense, es);
  if (!p.k_stride || !p.v_stride) return GDN_ERR_SHAPE;
  p.num_global = num_global_tokens;
  if (num_q_heads > 0) {
    const int64_t width = (int64_t)num_q_heads * cache->head_dim;
    p.q = q;
    p.q_out = q_out;
    p.q_stride = token_stride(q_stride, width, es);
    p.q_out_stride = token_stride(q_out_stride, width, es);
    if (!p.q_stride || !p.q_out_stride) return GDN_ERR_SHAPE;
    const int n = num_global_tokens;
    if (entangled(q, p.q_stride, width, q_out, p.q_out_stride, width, n, es, true) ||
        entangled(k, p.k_stride, dense, q_out, p.q_out_stride, width, n, es, false) ||
        entangled(v, p.v_stride, dense, q_out, p.q_out_stride, width, n, es, false))
      return GDN_ERR_SHAPE;
  }
  p.Hq = num_q_heads;
  p.d = cache->head_dim;
  p.num_tokens = rows->num_tokens;
  p.status = d_status;
  return cuda_rc(launch_kv_append_rope(p, cache->dtype, (cudaStream_t)stream));
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
  int rc = attention_checks(attn, cache, rows, q, num_global_tokens, out);
  if (rc || rows->num_tokens == 0) return rc;
  AttnLaunch p;
  if ((rc = attention_args(attn, cache, rows, q, q_stride, num_global_tokens, out, out_stride, workspace, workspace_bytes,
                           gdn_attention_workspace_bytes(attn, cache, rows), d_status, p)))
    return rc;
  return attend_whole(p, cache->dtype, (cudaStream_t)stream);
}

size_t gdn_shared_attention_workspace_bytes(const gdn_attn_desc* attn, const gdn_kv_cache* cache, const gdn_kv_rows* rows,
                                            const gdn_kv_groups* groups) {
  if (check_groups(groups)) return 0;
  const size_t whole = gdn_attention_workspace_bytes(attn, cache, rows);
  if (check_shape(cache) || check_table(cache) || check_attn(attn, cache) || check_kv_rows(rows)) return 0;
  AttnLaunch p = attn_args(attn, cache, rows);
  const Pass pass = pass_of(p, groups->num_groups, cache->dtype);
  if (pass == kNoPass) return whole;
  all_parts(p, groups->num_groups, pass);
  return shared_ws(p).end;
}

int gdn_shared_attention(const gdn_attn_desc* attn, const gdn_kv_cache* cache, const gdn_kv_rows* rows,
                         const gdn_kv_groups* groups, const void* q, int64_t q_stride, int32_t num_global_tokens, void* out,
                         int64_t out_stride, void* workspace, size_t workspace_bytes, uint32_t* d_status, void* stream) {
  Range range("gdn_shared_attention");
  int rc = attention_checks(attn, cache, rows, q, num_global_tokens, out);
  if (rc || (rc = check_groups(groups)) || rows->num_tokens == 0) return rc;
  const size_t need = gdn_shared_attention_workspace_bytes(attn, cache, rows, groups);
  AttnLaunch p;
  if ((rc = attention_args(attn, cache, rows, q, q_stride, num_global_tokens, out, out_stride, workspace, workspace_bytes,
                           need, d_status, p)))
    return rc;
  const Pass pass = pass_of(p, groups->num_groups, cache->dtype);
  if (pass == kNoPass) return attend_whole(p, cache->dtype, (cudaStream_t)stream);
  all_parts(p, groups->num_groups, pass);
  const SharedWs w = shared_ws(p);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  GroupsLaunch plan = groups_args(cache, rows, groups, d_status);
  plan.window = p.window;
  plan.sinks = p.sinks;
  plan.recs = reinterpret_cast<PartRec*>(ws + w.recs);
  plan.token = reinterpret_cast<int2*>(ws + w.token);
  p.part.recs = plan.recs;
  p.part.token = plan.token;
  p.part.start = plan.start;
  p.part.prefix = plan.prefix;
  p.part.range = reinterpret_cast<PieceRange*>(ws + w.range);
  p.part.ml = reinterpret_cast<float*>(ws + w.ml);
  p.part.o = reinterpret_cast<float*>(ws + w.o);
  p.ws = ws + w.pass;
  const cudaStream_t s = (cudaStream_t)stream;
  if (!p.part.plan_here && (rc = cuda_rc(launch_group_plan(plan, s)))) return rc;
  PartPieces pieces;
  if (pass == kTilePass) {
    pieces = attn_shared_pieces(p, p.ws);
    rc = cuda_rc(launch_attn_shared(p, s));
  } else {
    pieces = attn_split_fma_parts_pieces(p, p.ws);
    rc = cuda_rc(launch_attn_split_fma_parts(p, cache->dtype, s));
  }
  return rc ? rc : cuda_rc(launch_join_parts(p, cache->dtype, pieces, s));
}

int gdn_kv_common_prefix(const gdn_kv_cache* cache, const gdn_kv_rows* rows, const gdn_kv_groups* groups,
                         uint32_t* d_status, void* stream) {
  Range range("gdn_kv_common_prefix");
  int rc;
  if ((rc = check_shape(cache)) || (rc = check_table(cache)) || (rc = check_kv_rows(rows)) || (rc = check_groups(groups)))
    return rc;
  if (groups->num_groups == 0) return GDN_OK;
  return cuda_rc(launch_kv_common_prefix(groups_args(cache, rows, groups, d_status), (cudaStream_t)stream));
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
