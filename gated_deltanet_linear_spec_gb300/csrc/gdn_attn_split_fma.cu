// gdn_attn_split_fma.cu -- attention on the CUDA cores: 32-bit caches, and the head dimensions that the tensor core
// kernels do not take (bf16 with d other than 64, 128 and 256).
//
// The work is dealt out as in gdn_attn_split.cu; a worker is a warp, a unit 8 queries of a (row, kv-head), rows
// have any length.  Per 32 cached tokens a lane scores one token against the 8 queries in 32-bit FMAs, then the lanes
// turn to the output's columns, E neighbours each, and walk the tokens.  2 x 8 FMAs per pair of cached values are
// little, but every broadcast of a query's or weight's 16 bytes to a warp fills its registers in four cycles, and that
// bounds long caches; short ones are bound by the tiles' latency.  The values of a tile are fetched in batches
// before they are wanted (one token at a time: 67 us instead of 29 for 24 verify rows of 3 tokens, 8 q-heads, 2
// kv-heads, d = 64, 32 bits, contexts of 64 to 4096).  Tried and slower there: packed pairs of FMAs (34 us), 8 warps a
// CTA at 128 registers (spills), keys staged in shared memory (32 us).  1024 new tokens at 4096 take 545 us;
// with a warp per query, which shares nothing, 4190; 64 decode rows over 512 to 8192 tokens (bf16, d = 96, 32 q-heads,
// 4 kv-heads) 180 us against 5731.
// A tile's outputs are summed on their own and added once, which keeps long sums exact to a few steps.
#include <algorithm>

#include "gdn_attn_share.cuh"

namespace gdn {

namespace {

using namespace split;

constexpr int kWarps = 4;   // workers of a CTA
constexpr int kPerSm = 2;   // CTAs
constexpr int kNQ = 8;      // queries of a unit

template <typename T>
struct Vec {  // 16 bytes
  static constexpr int kN = 16 / sizeof(T);
};
// 16 bytes' values.
__device__ __forceinline__ void load16(const float* v, bool there, float (&x)[4]) {
  const float4 y = there ? __ldg(reinterpret_cast<const float4*>(v)) : make_float4(0.f, 0.f, 0.f, 0.f);
  x[0] = y.x;
  x[1] = y.y;
  x[2] = y.z;
  x[3] = y.w;
}
__device__ __forceinline__ void open2(uint32_t u, float& lo, float& hi) {
  lo = __uint_as_float(u << 16);
  hi = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ void load16(const __nv_bfloat16* v, bool there, float (&x)[8]) {
  const uint4 y = there ? __ldg(reinterpret_cast<const uint4*>(v)) : make_uint4(0, 0, 0, 0);
  open2(y.x, x[0], x[1]);
  open2(y.y, x[2], x[3]);
  open2(y.z, x[4], x[5]);
  open2(y.w, x[6], x[7]);
}
// E neighbouring values of a row, aligned to their size; zeros unless `there`.
template <int E>
__device__ __forceinline__ void load_row(const float* v, bool there, float (&x)[E]) {
  if constexpr (E == 1) {
    x[0] = there ? __ldg(v) : 0.f;
  } else if constexpr (E == 2) {
    const float2 y = there ? __ldg(reinterpret_cast<const float2*>(v)) : make_float2(0.f, 0.f);
    x[0] = y.x;
    x[1] = y.y;
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      float y[4];
      load16(v + e, there, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[e + i] = y[i];
    }
  }
}
template <int E>
__device__ __forceinline__ void load_row(const __nv_bfloat16* v, bool there, float (&x)[E]) {
  if constexpr (E == 2) {
    open2(there ? __ldg(reinterpret_cast<const uint32_t*>(v)) : 0u, x[0], x[1]);
  } else if constexpr (E == 4) {
    const uint2 y = there ? __ldg(reinterpret_cast<const uint2*>(v)) : make_uint2(0, 0);
    open2(y.x, x[0], x[1]);
    open2(y.y, x[2], x[3]);
  } else {
    load16(v, there, x);
  }
}

// E: columns of a lane, 32 E are head_dim or more; DC: head_dim where it is 32 E, else 0.
template <typename T, int E, int DC>
__global__ void __launch_bounds__(32 * kWarps, kPerSm) split_fma_kernel(SplitParams P) {
  constexpr int kU = E <= 2 ? 16 : E == 4 ? 8 : 2;  // tokens whose values a lane holds at a time
  constexpr int kV = Vec<T>::kN;
  __shared__ __align__(16) float sq[kWarps][kNQ][32 * E];
  __shared__ __align__(16) float sp[kWarps][32][kNQ];
  __shared__ int64_t part[kWarps];
  __shared__ Deal deal;
  __shared__ Share shares[kWarps];
  const AttnLaunch& p = P.a;
  const KvDev& kv = p.cache;
  const int D = DC > 0 ? DC : kv.d;  // a multiple of 16, so of E
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int worker = blockIdx.x * kWarps + warp;
  const bool columns = DC > 0 || lane * E < D;  // this lane has some
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (lane == 0) P.info[worker * 8] = 0;
  find_shares<kNQ, kWarps, 32 * kWarps>(p, part, deal, shares);
  const Share& share = shares[warp];
  const float sl2 = p.scale * 1.4426950408889634f;
  const int shift = __ffs(kv.page_size) - 1;

  for (Walk<kNQ> w(p, share); w.valid(); w.next()) {
    const KvRow row = w.u.r;
    const int h = w.h % kv.Hkv, q0 = w.h / kv.Hkv * kNQ, nq = min(kNQ, row.len * p.G - q0);
    const int first = row.kv - row.len;  // position of the first new token
    int g = -1;                          // lane i < nq: the query's global token
    if (lane < nq) g = global_token(RowsDev{nullptr, p.rows.tok}, row.bos + (q0 + lane) / p.G, p.num_global, p.status);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kNQ; ++i) {
      const int gi = __shfl_sync(0xffffffffu, g, i);
      const T* q =
          static_cast<const T*>(p.q) + (int64_t)max(gi, 0) * p.q_stride + (int64_t)(h * p.G + (q0 + i) % p.G) * D;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = lane + 32 * e;
        sq[warp][i][c] = gi >= 0 && (DC > 0 || c < D) ? to_f32(q[c]) : 0.f;
      }
    }
    __syncwarp();
    const int pos0 = first + q0 / p.G, pos1 = first + (q0 + nq - 1) / p.G;  // of the first and last query
    float o[kNQ][E], m[kNQ], l[kNQ];
#pragma unroll
    for (int i = 0; i < kNQ; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[i][e] = 0.f;
    }
    const int32_t* table = kv.table + (int64_t)row.trow * kv.max_pages;
    auto entry = [&](int j) {  // the table's entry of this lane's token of tile j
      const int tok = w.tile_at(j) + lane;
      return j < w.j0 + w.len && tok <= pos1 ? __ldg(table + (tok >> shift)) : 0;
    };
    int ahead = entry(w.j0);
    for (int j = w.j0; j < w.j0 + w.len; ++j) {
      const int b = w.tile_at(j), tok = b + lane;
      const int page = page_or_null(ahead, kv, p.status);
      ahead = entry(j + 1);
      // some query sees this lane's token
      const bool some = page > 0 && (p.window <= 0 || tok > pos0 - p.window || tok < p.sinks);
      const unsigned seen = __ballot_sync(0xffffffffu, some);
      if (seen == 0) continue;
      const int64_t at = (int64_t)page * kv.page_stride + ((int64_t)h * kv.page_size + (tok & (kv.page_size - 1))) * D;
      // the values of kU tokens, a lane per E columns, on their way while those before are worked on; a page holds
      // 16 tokens or more
      float x[2][kU][E];
      auto fetch = [&](int c) {
        const T* v = static_cast<const T*>(kv.v) + __shfl_sync(0xffffffffu, at, c * kU & 16) + lane * E;
#pragma unroll
        for (int u = 0; u < kU; ++u)
          load_row<E>(v + (int64_t)(c * kU % 16 + u) * D, columns && (seen >> (c * kU + u) & 1u), x[c & 1][u]);
      };
      fetch(0);
      float s[kNQ];
#pragma unroll
      for (int i = 0; i < kNQ; ++i) s[i] = 0.f;
      const T* k = static_cast<const T*>(kv.k) + at;
#pragma unroll(DC > 0 ? 16 : 4)
      for (int c = 0; c < D; c += kV) {
        float y[kV];
        load16(k + c, some, y);
#pragma unroll
        for (int i = 0; i < kNQ; ++i)
#pragma unroll
          for (int e = 0; e < kV; e += 4) {
            const float4 q = *reinterpret_cast<const float4*>(&sq[warp][i][c + e]);
            s[i] = fmaf(q.x, y[e], fmaf(q.y, y[e + 1], fmaf(q.z, y[e + 2], fmaf(q.w, y[e + 3], s[i]))));
          }
      }
      float f[kNQ];
#pragma unroll
      for (int i = 0; i < kNQ; ++i) {
        const int pos = min(first + (q0 + i) / p.G, pos1);
        const bool sees = some && tok <= pos && (p.window <= 0 || tok > pos - p.window || tok < p.sinks);
        if (!sees) s[i] = -INFINITY;
        float x = s[i];
#pragma unroll
        for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
        const float mn = fmaxf(m[i], x);
        f[i] = m[i] == -INFINITY ? 0.f : ex2((m[i] - mn) * sl2);
        m[i] = mn;
        const float e = ex2(fmaf(s[i], sl2, mn == -INFINITY ? 0.f : -mn * sl2));
        l[i] = l[i] * f[i] + e;
        sp[warp][lane][i] = e;
      }
      __syncwarp();
      // the tile's own sums, a lane per E columns; a weight of 0 takes no value in, whatever that holds
      float t[kNQ][E];
#pragma unroll
      for (int i = 0; i < kNQ; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) t[i][e] = 0.f;
#pragma unroll
      for (int c = 0; c < 32 / kU; ++c) {
        if (c + 1 < 32 / kU) fetch(c + 1);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          float pw[kNQ];
          *reinterpret_cast<float4*>(pw) = *reinterpret_cast<const float4*>(&sp[warp][c * kU + u][0]);
          *reinterpret_cast<float4*>(pw + 4) = *reinterpret_cast<const float4*>(&sp[warp][c * kU + u][4]);
#pragma unroll
          for (int i = 0; i < kNQ; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) t[i][e] = pw[i] == 0.f ? t[i][e] : fmaf(pw[i], x[c & 1][u][e], t[i][e]);
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kNQ; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) o[i][e] = fmaf(o[i][e], f[i], t[i][e]);
    }

    const bool whole = w.j0 == 0 && w.len == w.u.tiles;
    const int slot = 2 * worker + (w.j0 == 0 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < kNQ; ++i) {
#pragma unroll
      for (int d = 16; d; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      const int gi = __shfl_sync(0xffffffffu, g, i);
      if (i >= nq) continue;
      if (whole) {
        if (gi < 0) continue;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        T* out = static_cast<T*>(p.out) + (int64_t)gi * p.out_stride + (int64_t)(h * p.G + (q0 + i) % p.G) * D;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (columns) out[lane * E + e] = from_f32<T>(o[i][e] * inv);
      } else {
        float* dst = P.part + ((size_t)slot * kNQ + i) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (columns) dst[e] = o[i][e];
        if (lane == 0)
          *reinterpret_cast<float2*>(P.stats + ((size_t)slot * kNQ + i) * 2) = make_float2(m[i], l[i]);
      }
    }
    if (!whole && w.j0 == 0 && lane == 0) {
      int32_t* info = P.info + worker * 8;
      info[1] = row.bos;
      info[2] = nq;
      info[3] = h;
      info[4] = deal.owner(w.unit_last(share));  // the worker with the unit's last tile
      info[5] = q0;
      info[0] = 1;
    }
  }
}

template <typename T, int E, int DC>
cudaError_t launch_as(const AttnLaunch& a, cudaStream_t s) {
  constexpr int ctas = kSms * kPerSm;
  SplitParams P{};
  P.a = a;
  P.info = static_cast<int32_t*>(a.ws);
  P.stats = reinterpret_cast<float*>(P.info + 8 * ctas * kWarps);
  P.part = P.stats + (size_t)4 * ctas * kWarps * kNQ;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, split_fma_kernel<T, E, DC>, P);
  if (e != cudaSuccess) return e;
  const int queries = (int)std::min<int64_t>(kNQ, (int64_t)a.rows.max_q * a.G);
  cfg.gridDim = dim3(ctas * kWarps, join_rows(ctas * kWarps, queries));
  cfg.blockDim = dim3(32 * kJoinWarps);
  return cudaLaunchKernelEx(&cfg, join_kernel<T, E, DC>, P, kNQ);
}
template <typename T>
cudaError_t launch_any(const AttnLaunch& a, cudaStream_t s) {
  const int d = a.cache.d;
  return d <= 64 ? launch_as<T, 2, 0>(a, s) : d <= 128 ? launch_as<T, 4, 0>(a, s) : launch_as<T, 8, 0>(a, s);
}

}  // namespace

size_t attn_split_fma_workspace(const AttnLaunch& a) {
  return (size_t)kSms * kPerSm * kWarps * (8 + 4 * kNQ + 2 * kNQ * a.cache.d) * 4;
}

cudaError_t launch_attn_split_fma(const AttnLaunch& a, gdn_dtype dtype, cudaStream_t s) {
  if (dtype == GDN_BF16) return launch_any<__nv_bfloat16>(a, s);
  switch (a.cache.d) {
    case 32: return launch_as<float, 1, 32>(a, s);
    case 64: return launch_as<float, 2, 64>(a, s);
    case 128: return launch_as<float, 4, 128>(a, s);
    case 256: return launch_as<float, 8, 256>(a, s);
    default: return launch_any<float>(a, s);
  }
}

}  // namespace gdn
