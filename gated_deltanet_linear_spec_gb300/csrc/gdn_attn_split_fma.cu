// gdn_attn_split_fma.cu -- attention on the CUDA cores: 32-bit caches, and the head dimensions that the tensor core
// kernels do not take (bf16 with d other than 64, 128 and 256).
//
// The work is dealt out as in gdn_attn_split.cu; a worker is a warp, a unit 8 queries of a (row, kv-head), rows
// have any length.  A lane holds E neighbouring columns of the 8 queries and of their outputs in registers and walks
// the keys, then the values, of 32 tokens a step: 2 x 8 32-bit FMAs per pair of cached values.  The parts of 8 x 4
// scores meet by exchanges that halve what a lane keeps, so a lane ends up with one query's scores of every fourth
// token, and the softmax takes two exchanges.  (Scores by lane = token, queries broadcast from shared memory, are
// bound by those broadcasts, four cycles each: 64 rows of 3 tokens, 64 to 4096 cached, 8 q-heads, 2 kv-heads, 32 bits,
// d = 256: 187 us instead of 126.)  Keys and values are fetched a chunk ahead; one token at a time, 24 such rows
// with d = 64 took 67 us instead of 26.  Loops of two chunks a turn, as unrolled ones fall out of the instruction
// cache (d = 96: 1467 us instead of 714 for 1024 new tokens at 2048, 16 q-heads, 4 kv-heads).
// Per token of a step, a unit of 8 queries takes about 16 E FMAs and 8 exchanges: that bounds long caches, the
// steps' latency short ones.  1024 new tokens at 4096 (d = 64) take 432 us, with a warp per query, which shares
// nothing, 4190; 64 decode rows over 512 to 8192 tokens (bf16, d = 96, 32 q-heads, 4 kv-heads) 198 us against 5731.
// Up to d = 128 a step's outputs are summed on their own and added once, which keeps long sums exact to a few steps.
#include <algorithm>

#include "gdn_attn_share.cuh"

namespace gdn {

namespace {

using namespace split;

constexpr int kWarps = 4;   // workers of a CTA
constexpr int kPerSm = 2;   // CTAs
constexpr int kNQ = 8;      // queries of a unit

// 16 bytes' values.
__device__ __forceinline__ void load16(const float* v, bool there, float (&x)[4]) {
  const float4 y = there ? load(reinterpret_cast<const float4*>(v)) : make_float4(0.f, 0.f, 0.f, 0.f);
  x[0] = y.x;
  x[1] = y.y;
  x[2] = y.z;
  x[3] = y.w;
}
__device__ __forceinline__ void open2(uint32_t u, float& lo, float& hi) {
  lo = __uint_as_float(u << 16);
  hi = __uint_as_float(u & 0xffff0000u);
}
// (Eight columns a lane: a load that keeps its place.  Plain ones are moved ahead and 232 bytes of registers spill: 1024
// new tokens at 2048, d = 192, 16 q-heads, 4 kv-heads 1162 us instead of 1061.  At d = 96 plain ones win, 196 and 203 us
// for 64 decode rows.)
__device__ __forceinline__ void load16(const __nv_bfloat16* v, bool there, float (&x)[8]) {
  const uint4 y = there ? __ldca(reinterpret_cast<const uint4*>(v)) : make_uint4(0, 0, 0, 0);
  open2(y.x, x[0], x[1]);
  open2(y.y, x[2], x[3]);
  open2(y.z, x[4], x[5]);
  open2(y.w, x[6], x[7]);
}
// E neighbouring values of a row, aligned to their size; zeros unless `there`.
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
    open2(there ? load(reinterpret_cast<const uint32_t*>(v)) : 0u, x[0], x[1]);
  } else if constexpr (E == 4) {
    const uint2 y = there ? load(reinterpret_cast<const uint2*>(v)) : make_uint2(0, 0);
    open2(y.x, x[0], x[1]);
    open2(y.y, x[2], x[3]);
  } else {
    load16(v, there, x);
  }
}

// E: columns of a lane, 32 E are head_dim or more; DC: head_dim where it is 32 E, else 0.
template <typename T, int E, int DC>
__global__ void __launch_bounds__(32 * kWarps, kPerSm) split_fma_kernel(SplitParams P) {
  constexpr int kU = E <= 4 ? 8 : 4;  // tokens whose keys or values a lane holds at a time
  constexpr int kC = 32 / kU;         // as many chunks of keys, then as many of values
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
    if (lane < nq) g = kv_token(p.rows, row.bos + (q0 + lane) / p.G, p.num_global, p.status);
    float q[kNQ][E];
#pragma unroll
    for (int i = 0; i < kNQ; ++i) {
      const int gi = __shfl_sync(0xffffffffu, g, i);
      const T* from = static_cast<const T*>(p.q) + (int64_t)max(gi, 0) * p.q_stride;
      load_row<E>(from + (int64_t)(h * p.G + (q0 + i) % p.G) * D + lane * E, columns && gi >= 0, q[i]);
    }
    const int pos0 = first + q0 / p.G, pos1 = first + (q0 + nq - 1) / p.G;  // of the first and last query
    const int mine = lane >> 2;  // the query whose scores, maximum and sum this lane has, those of every 4th token
    const int pos = min(first + (q0 + mine) / p.G, pos1);
    float o[kNQ][E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < kNQ; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) o[i][e] = 0.f;
    const int32_t* table = kv.table + (int64_t)row.trow * kv.max_pages;
    auto entry = [&](int j) {  // the table's entry of this lane's token of tile j
      const int tok = w.tile_at(j) + lane;
      return j < w.j0 + w.len && tok <= pos1 ? load(table + (tok >> shift)) : 0;
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
      // chunk c of the keys, then of the values, on its way while the one before is worked on; a page holds 16 tokens
      // or more
      float x[2][kU][E];
      auto fetch = [&](int c, float (&to)[kU][E]) {
        const int from = c % kC * kU;
        const T* v = static_cast<const T*>(c < kC ? kv.k : kv.v) + __shfl_sync(0xffffffffu, at, from & 16) +
                     from % 16 * D + lane * E;
#pragma unroll
        for (int u = 0; u < kU; ++u) load_row<E>(v + u * D, columns && (seen >> (from + u) & 1u), to[u]);
      };
      fetch(0, x[0]);
      // (rolled, two chunks a turn: in one piece these loops are too long for the instruction cache)
#pragma unroll 1
      for (int c0 = 0; c0 < kC; c0 += 2) {
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const int c = c0 + d;
          fetch(c + 1, x[d ^ 1]);
#pragma unroll
          for (int n = 0; n < kU / 4; ++n) {
            // A lane's part of 8 queries x 4 tokens; halving what a lane keeps with every exchange, 31 of them leave it
            // the sum of one.
            float r[32];
#pragma unroll
            for (int i = 0; i < kNQ; ++i)
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                float t = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) t = fmaf(q[i][e], x[d][4 * n + u][e], t);
                r[4 * i + u] = t;
              }
#pragma unroll
            for (int half = 16; half; half >>= 1)
#pragma unroll
              for (int i = 0; i < half; ++i) {
                const float keep = lane & half ? r[i + half] : r[i], give = lane & half ? r[i] : r[i + half];
                r[i] = keep + __shfl_xor_sync(0xffffffffu, give, half);
              }
            sp[warp][c * kU + 4 * n + (lane & 3)][mine] = r[0];
          }
        }
      }
      float s[8];  // of tokens (lane & 3) + 4 n, which this lane wrote
#pragma unroll
      for (int n = 0; n < 8; ++n) s[n] = sp[warp][4 * n + (lane & 3)][mine];
      float x_max = -INFINITY;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int t = 4 * n + (lane & 3), tk = b + t;
        const bool sees = (seen >> t & 1u) && tk <= pos && (p.window <= 0 || tk > pos - p.window || tk < p.sinks);
        if (!sees) s[n] = -INFINITY;
        x_max = fmaxf(x_max, s[n]);
      }
      x_max = fmaxf(x_max, __shfl_xor_sync(0xffffffffu, x_max, 1));
      x_max = fmaxf(x_max, __shfl_xor_sync(0xffffffffu, x_max, 2));
      const float mn = fmaxf(m, x_max);
      const float f = m == -INFINITY ? 0.f : ex2((m - mn) * sl2);
      const float ms = mn == -INFINITY ? 0.f : -mn * sl2;
      m = mn;
      l *= f;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float e = ex2(fmaf(s[n], sl2, ms));
        l += e;
        sp[warp][4 * n + (lane & 3)][mine] = e;
      }
      __syncwarp();
      // The tile's own sums (with 8 columns a lane there are no registers for them); a weight of 0 takes no value in,
      // whatever that holds.
      constexpr bool kOwn = E <= 4;
      float t[kNQ][E];
#pragma unroll
      for (int i = 0; i < kNQ; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, 4 * i);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          t[i][e] = kOwn ? 0.f : o[i][e] * fi;
          if (kOwn) o[i][e] *= fi;
        }
      }
#pragma unroll 1
      for (int c0 = 0; c0 < kC; c0 += 2) {
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const int c = c0 + d;
          if (c + 1 < kC) fetch(kC + c + 1, x[d ^ 1]);
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            float pw[kNQ];
            *reinterpret_cast<float4*>(pw) = *reinterpret_cast<const float4*>(&sp[warp][c * kU + u][0]);
            *reinterpret_cast<float4*>(pw + 4) = *reinterpret_cast<const float4*>(&sp[warp][c * kU + u][4]);
#pragma unroll
            for (int i = 0; i < kNQ; ++i)
#pragma unroll
              for (int e = 0; e < E; ++e) t[i][e] = pw[i] == 0.f ? t[i][e] : fmaf(pw[i], x[d][u][e], t[i][e]);
          }
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kNQ; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) o[i][e] = kOwn ? o[i][e] + t[i][e] : t[i][e];
    }

    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const bool whole = w.j0 == 0 && w.len == w.u.tiles;
    const int slot = 2 * worker + (w.j0 == 0 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < kNQ; ++i) {
      const float li = __shfl_sync(0xffffffffu, l, 4 * i), mi = __shfl_sync(0xffffffffu, m, 4 * i);
      const int gi = __shfl_sync(0xffffffffu, g, i);
      if (i >= nq) continue;
      if (whole) {
        if (gi < 0) continue;
        const float inv = li == 0.f ? 0.f : 1.f / li;
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
          *reinterpret_cast<float2*>(P.stats + ((size_t)slot * kNQ + i) * 2) = make_float2(mi, li);
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
  const int queries = (int)std::min<int64_t>(kNQ, std::max<int64_t>(1, (int64_t)a.rows.max_q * a.G));
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
