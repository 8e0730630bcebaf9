// gdn_attn_scalar.cu -- attention over the paged cache for every layout, on the CUDA cores.
//
// A warp owns one query (token, q-head) and walks the keys that it sees, lanes over the head
// dimension: score by a warp sum, then the running maximum m, sum l and output o of the softmax,
//   m' = max(m, s), o <- o e^(m-m') + e^(s-m') v, l <- l e^(m-m') + e^(s-m').
// Keys that the query does not see are never loaded.
#include "gdn_kv.cuh"

namespace gdn {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxPer = 8;  // head_dim <= 256

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) attn_scalar_kernel(AttnLaunch p) {
  const KvDev& C = p.cache;
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int local = (int)(id / p.Hq), h = (int)(id - (int64_t)local * p.Hq);
  if (local >= p.rows.num_tokens) return;
  int lo = 0, hi = p.rows.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.rows.qsl + mid) <= local) lo = mid; else hi = mid - 1;
  }
  KvRow r;
  if (!load_kv_row(p.rows, C, lo, r, p.status) || local < r.bos || local >= r.bos + r.len) return;
  const int32_t g = p.rows.tok ? __ldg(p.rows.tok + local) : local;
  if (g < 0 || g >= p.num_global) {
    set_status(p.status, GDN_STATUS_TOKEN_RANGE);
    return;
  }
  const int pos = r.kv - r.len + (local - r.bos);
  const int per = (C.d + 31) / 32;
  const T* q = static_cast<const T*>(p.q) + (int64_t)g * p.q_stride + (int64_t)h * C.d;
  float qv[kMaxPer], o[kMaxPer];
#pragma unroll
  for (int i = 0; i < kMaxPer; ++i) {
    const int e = lane + 32 * i;
    qv[i] = i < per && e < C.d ? to_f32(q[e]) * p.scale : 0.f;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int32_t* row = C.table + (int64_t)r.trow * C.max_pages;
  const int first = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  const int sinks = min(p.sinks, first);
  const int64_t head = (int64_t)(h / p.G) * C.page_size * C.d;
  for (int j = sinks > 0 ? 0 : first; j <= pos;) {
    const int page = page_or_null(row[j / C.page_size], C, p.status);
    int end = min((j / C.page_size + 1) * C.page_size, pos + 1);
    if (j < sinks) end = min(end, sinks);
    if (page > 0) {
      const int64_t off = (int64_t)page * C.page_stride + head + (int64_t)(j % C.page_size) * C.d;
      const T* k = static_cast<const T*>(C.k) + off;
      const T* v = static_cast<const T*>(C.v) + off;
      for (int t = j; t < end; ++t, k += C.d, v += C.d) {
        float s = 0.f, vv[kMaxPer];
#pragma unroll
        for (int i = 0; i < kMaxPer; ++i) {
          const int e = lane + 32 * i;
          const bool in = i < per && e < C.d;
          s += in ? qv[i] * to_f32(k[e]) : 0.f;
          vv[i] = in ? to_f32(v[e]) : 0.f;
        }
#pragma unroll
        for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        const float m2 = fmaxf(m, s);
        const float a = m == m2 ? 1.f : expf(m - m2), e = expf(s - m2);
        l = l * a + e;
#pragma unroll
        for (int i = 0; i < kMaxPer; ++i) o[i] = o[i] * a + e * vv[i];
        m = m2;
      }
    }
    j = end;
    if (j == sinks && j < first) j = first;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = static_cast<T*>(p.out) + (int64_t)g * p.out_stride + (int64_t)h * C.d;
#pragma unroll
  for (int i = 0; i < kMaxPer; ++i) {
    const int e = lane + 32 * i;
    if (i < per && e < C.d) out[e] = from_f32<T>(o[i] * inv);
  }
}

}  // namespace

cudaError_t launch_attn_scalar(const AttnLaunch& p, gdn_dtype dtype, cudaStream_t s) {
  const int64_t warps = (int64_t)p.rows.num_tokens * p.Hq;
  const int blocks = (int)((warps + kWarps - 1) / kWarps);
  if (dtype == GDN_BF16)
    attn_scalar_kernel<__nv_bfloat16><<<blocks, kWarps * 32, 0, s>>>(p);
  else
    attn_scalar_kernel<float><<<blocks, kWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
