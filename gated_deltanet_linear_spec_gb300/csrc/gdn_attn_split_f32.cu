// gdn_attn_split_f32.cu -- attention over a 32-bit cache (d = 32, 64, 128, 256).
//
// The work is dealt out as in gdn_attn_split.cu; a worker is a warp, a unit 8 queries of a (row, kv-head).
// Products are 32-bit FMAs (the tensor cores have no such type): per 32 cached tokens a lane scores one token
// against the 8 queries, then the lanes turn to the output's columns and walk the tokens.  2 x 8 FMAs
// per pair of cached floats are little, but every broadcast of a query's or weight's 16 bytes to a warp fills its
// registers in four cycles, and that bounds long caches; short ones are bound by the tiles' latency.  The values of a
// tile are fetched in batches before they are wanted (one token at a time: 67 us instead of 29 for 24
// verify rows of 3 tokens, 8 q-heads, 2 kv-heads, d = 64, contexts of 64 to 4096).  Tried and slower there: packed
// pairs of FMAs (34 us), 8 warps a CTA at 128 registers (spills), keys staged in shared memory (32 us).
// Rows of any length come here: eight queries share every key and value (1024 new tokens at 4096, 8 q-heads, d = 64:
// 545 us; a warp per query, as in gdn_attn_scalar.cu, 4190).
// A tile's outputs are summed on their own and added once, which keeps long sums exact to a few steps.
#include <algorithm>

#include "gdn_attn_share.cuh"

namespace gdn {

namespace {

using namespace split;

constexpr int kWarps = 4;   // workers of a CTA
constexpr int kPerSm = 2;   // CTAs
constexpr int kNQ = 8;      // queries of a unit

// E floats of a row, aligned to their size; zeros unless `there`.
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
      const float4 y = there ? __ldg(reinterpret_cast<const float4*>(v + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[e] = y.x;
      x[e + 1] = y.y;
      x[e + 2] = y.z;
      x[e + 3] = y.w;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps, kPerSm) split_f32_kernel(SplitParams P) {
  constexpr int E = D / 32;                          // output columns of a lane
  constexpr int kU = E <= 2 ? 16 : E == 4 ? 8 : 2;   // tokens whose values a lane holds at a time
  __shared__ __align__(16) float sq[kWarps][kNQ][D];
  __shared__ __align__(16) float sp[kWarps][32][kNQ];
  __shared__ int64_t part[kWarps];
  __shared__ Deal deal;
  __shared__ Share shares[kWarps];
  const AttnLaunch& p = P.a;
  const KvDev& kv = p.cache;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int worker = blockIdx.x * kWarps + warp;
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
      const float* q = static_cast<const float*>(p.q) + (int64_t)max(gi, 0) * p.q_stride + (int64_t)(h * p.G + (q0 + i) % p.G) * D;
#pragma unroll
      for (int e = 0; e < E; ++e) sq[warp][i][lane + 32 * e] = gi >= 0 ? __ldg(q + lane + 32 * e) : 0.f;
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
        const float* v = static_cast<const float*>(kv.v) + __shfl_sync(0xffffffffu, at, c * kU & 16) + lane * E;
#pragma unroll
        for (int u = 0; u < kU; ++u)
          load_row<E>(v + (int64_t)(c * kU % 16 + u) * D, seen >> (c * kU + u) & 1u, x[c & 1][u]);
      };
      fetch(0);
      float s[kNQ];
#pragma unroll
      for (int i = 0; i < kNQ; ++i) s[i] = 0.f;
      const float4* k = reinterpret_cast<const float4*>(static_cast<const float*>(kv.k) + at);
#pragma unroll 16
      for (int c = 0; c < D / 4; ++c) {
        const float4 y = some ? __ldg(k + c) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kNQ; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(&sq[warp][i][4 * c]);
          s[i] = fmaf(q.x, y.x, fmaf(q.y, y.y, fmaf(q.z, y.z, fmaf(q.w, y.w, s[i]))));
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
        float* out = static_cast<float*>(p.out) + (int64_t)gi * p.out_stride + (int64_t)(h * p.G + (q0 + i) % p.G) * D;
#pragma unroll
        for (int e = 0; e < E; ++e) out[lane * E + e] = o[i][e] * inv;
      } else {
        float* dst = P.part + ((size_t)slot * kNQ + i) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) dst[e] = o[i][e];
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

template <int D>
cudaError_t launch_d(const AttnLaunch& a, cudaStream_t s) {
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, split_f32_kernel<D>, P);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(ctas * kWarps, join_rows(ctas * kWarps, std::min(kNQ, a.rows.max_q * a.G)));
  cfg.blockDim = dim3(32 * kJoinWarps);
  return cudaLaunchKernelEx(&cfg, join_kernel<D, float>, P, kNQ);
}

}  // namespace

bool attn_split_f32_supported(const AttnLaunch& a, gdn_dtype dtype) {
  const int d = a.cache.d;
  return dtype == GDN_F32 && (d == 32 || d == 64 || d == 128 || d == 256);
}

size_t attn_split_f32_workspace(const AttnLaunch& a) {
  return (size_t)kSms * kPerSm * kWarps * (8 + 4 * kNQ + 2 * kNQ * a.cache.d) * 4;
}

cudaError_t launch_attn_split_f32(const AttnLaunch& a, cudaStream_t s) {
  switch (a.cache.d) {
    case 32: return launch_d<32>(a, s);
    case 64: return launch_d<64>(a, s);
    case 128: return launch_d<128>(a, s);
    case 256: return launch_d<256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gdn
