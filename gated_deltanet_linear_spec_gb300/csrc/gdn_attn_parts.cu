// gdn_attn_parts.cu -- joins what passes over parts of the rows' caches have left of every query.
//
// A query's result over one part is whole, or in pieces by the workers that shared its unit; over its group's shared tokens
// and its row's own ones together: m = max m_i, l = sum l_i e^(m_i - m), out = sum o_i e^(m_i - m) / l, the pieces in a fixed
// order.  A warp per query, or a team of them where queries are few and their pieces many (4 rows of 16 heads over 777 tokens:
// 12.1 us a call with teams, 16.2 without): a lane per piece for the statistics, then eight pieces' values on their way at a
// time.  What bounds it is that chain of loads; its bytes, (2 + d) fp32 per piece, lie in the L2.
#include <algorithm>

#include "gdn_attn_share.cuh"

namespace gdn {

namespace {

constexpr int kWarps = 8;

struct JoinParams {
  AttnLaunch a;
  PartPieces from;
  int team;  // warps of a query
};

// Whether a range names pieces that there are: one that a pass did not write, because a wait of it gave up, holds whatever the
// workspace held before.
__device__ __forceinline__ bool names_pieces(const PieceRange& r, const PartPieces& of) {
  return r.c0 < 0 || (r.c0 <= r.c1 && r.c1 < of.workers && r.qi >= 0 && r.qi < of.queries);
}

template <int E>
__device__ __forceinline__ void load_row(const float* v, bool there, float (&x)[E]) {
  if constexpr (E == 1) {
    x[0] = there ? load(v) : 0.f;
  } else if constexpr (E == 2) {
    const float2 y = there ? load(reinterpret_cast<const float2*>(v)) : make_float2(0.f, 0.f);
    x[0] = y.x;
    x[1] = y.y;
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const float4 y = there ? load(reinterpret_cast<const float4*>(v + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[e] = y.x;
      x[e + 1] = y.y;
      x[e + 2] = y.z;
      x[e + 3] = y.w;
    }
  }
}

// E columns of a lane; DC: head_dim where it is 32 E, else 0; QUADS: see PartDev.
template <typename T, int E, int DC, bool QUADS>
__global__ void __launch_bounds__(32 * kWarps) join_parts_kernel(JoinParams J) {
  constexpr int kAtOnce = E <= 4 ? 8 : 4;
  __shared__ float so[kWarps][32 * E], sl[kWarps], sm[kWarps];
  const AttnLaunch& p = J.a;
  const PartDev& part = p.part;
  const int D = DC > 0 ? DC : p.cache.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool columns = DC > 0 || lane * E < D;
  const float sl2 = p.scale * 1.4426950408889634f;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t all = (int64_t)part.tokens * p.Hq, q = (int64_t)blockIdx.x * (kWarps / J.team) + warp / J.team;
  const int token = q < all ? (int)((uint32_t)q / (uint32_t)p.Hq) : 0;  // (a call has fewer than 2^31 queries)
  int2 rec = make_int2(-1, 0);
  PieceRange r[2] = {};
  int g = -1;
  if (q < all) {
    rec = load(part.token + token);
    g = p.rows.tok ? load(p.rows.tok + token) : token;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int4 x = load(reinterpret_cast<const int4*>(part.range + s * all + q));
      r[s] = {x.x, x.y, x.z, 0};
    }
  }
  const bool there = rec.x >= 0 && g >= 0 && g < p.num_global && (!rec.y || names_pieces(r[0], J.from)) &&
                     names_pieces(r[1], J.from);
  const int n0 = !there || !rec.y ? 0 : r[0].c0 < 0 ? 1 : r[0].c1 - r[0].c0 + 1;
  const int n = !there ? 0 : n0 + (r[1].c0 < 0 ? 1 : r[1].c1 - r[1].c0 + 1);
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.f;
  for (int s0 = warp % J.team; s0 < n; s0 += 32 * J.team) {
    // a lane per piece: every team-th from s0 on
    const int i = s0 + lane * J.team, s = i < n0 ? 0 : 1;
    float2 st = make_float2(-INFINITY, 0.f);
    const float* values = nullptr;
    if (i < n) {
      const PieceRange x = s ? r[1] : r[0];
      const int c = x.c0 + i - (s ? n0 : 0);
      const int64_t at = x.c0 < 0 ? s * all + q : (int64_t)(2 * c + (c == x.c0 ? 1 : 0)) * J.from.queries + x.qi;
      st = load(reinterpret_cast<const float2*>(x.c0 < 0 ? part.ml : J.from.stats) + at);
      if (QUADS)
        values = x.c0 < 0 ? part.o + at * 4 : J.from.o + ((at - x.qi) * (D / 4) + x.qi) * 4;
      else
        values = (x.c0 < 0 ? part.o : J.from.o) + at * D;
    }
    float mn = st.x;
#pragma unroll
    for (int d = 16; d; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
    mn = fmaxf(mn, m);
    const float a = m == -INFINITY ? 0.f : split::ex2((m - mn) * sl2);
    const float f = st.x == -INFINITY ? 0.f : split::ex2((st.x - mn) * sl2);
    const int step = i < n && (s ? r[1].c0 : r[0].c0) < 0 ? (int)(2 * all) : J.from.queries;  // QUADS: 16 bytes from one to the next
    float sum = st.y * f;
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    l = l * a + sum;
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= a;
    const int mine = min(32, (n - s0 + J.team - 1) / J.team);
    for (int u0 = 0; u0 < mine; u0 += kAtOnce) {
      float v[kAtOnce][E];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const uint64_t from = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(values), (u0 + u) & 31);
        if constexpr (QUADS) {
          const int64_t to = __shfl_sync(0xffffffffu, step, (u0 + u) & 31);
          const float* x = reinterpret_cast<const float*>(from) + lane * E / 4 * to * 4 + lane * E % 4;
          if constexpr (E <= 4) {
            load_row<E>(x, u0 + u < mine, v[u]);
          } else {
#pragma unroll
            for (int e = 0; e < E; e += 4) {
              float y[4];
              load_row<4>(x + e * to, u0 + u < mine, y);
#pragma unroll
              for (int k = 0; k < 4; ++k) v[u][e + k] = y[k];
            }
          }
        } else {
          load_row<E>(reinterpret_cast<const float*>(from) + lane * E, u0 + u < mine && columns, v[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const float b = __shfl_sync(0xffffffffu, f, (u0 + u) & 31);
        if (u0 + u < mine) {
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = fmaf(v[u][e], b, o[e]);
        }
      }
    }
  }
  if (J.team > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
    __syncthreads();
    if (warp % J.team) return;
    for (int v = warp + 1; v < warp + J.team; ++v) {
      const float mn = fmaxf(m, sm[v]);
      const float a = m == -INFINITY ? 0.f : split::ex2((m - mn) * sl2);
      const float b = sm[v] == -INFINITY ? 0.f : split::ex2((sm[v] - mn) * sl2);
      l = l * a + sl[v] * b;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * a + so[v][lane + 32 * e] * b;
      m = mn;
    }
  }
  if (!there || !columns) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = static_cast<T*>(p.out) + (int64_t)g * p.out_stride + (q - (int64_t)token * p.Hq) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = from_f32<T>(o[e] * inv);
}

template <typename T, int E, int DC, bool QUADS>
cudaError_t launch_as(JoinParams& J, cudaStream_t s) {
  const int64_t queries = (int64_t)J.a.part.tokens * J.a.Hq;
  J.team = 8;
  while (J.team > 1 && queries * J.team > kSms * 32) J.team /= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int per = kWarps / J.team;
  cfg.gridDim = dim3((unsigned)((queries + per - 1) / per));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_parts_kernel<T, E, DC, QUADS>, J);
}
template <typename T>
cudaError_t launch_rows(JoinParams& J, cudaStream_t s) {
  const int d = J.a.cache.d;
  return d <= 64    ? launch_as<T, 2, 0, false>(J, s)
         : d <= 128 ? launch_as<T, 4, 0, false>(J, s)
                    : launch_as<T, 8, 0, false>(J, s);
}

}  // namespace

cudaError_t launch_join_parts(const AttnLaunch& p, gdn_dtype dtype, PartPieces pieces, cudaStream_t s) {
  JoinParams J{p, pieces, 1};
  if (dtype == GDN_F32) return launch_rows<float>(J, s);
  if (!p.part.quads) return launch_rows<__nv_bfloat16>(J, s);
  const int d = p.cache.d;
  return d == 64    ? launch_as<__nv_bfloat16, 2, 64, true>(J, s)
         : d == 128 ? launch_as<__nv_bfloat16, 4, 128, true>(J, s)
                    : launch_as<__nv_bfloat16, 8, 256, true>(J, s);
}

}  // namespace gdn
