// gdn_kv_rope.cu -- rotary positions: heads turned by their tokens' positions, alone or on their way into the cache.
//
// Pair i of a head's first r = rotary_dim values is (x_i, x_{i+r/2}) or (x_2i, x_2i+1); at position p it turns by the
// angle p f_i.  Frequencies are 64-bit fractions of a turn, so p f_i mod 1 is a product of whole numbers that wraps
// around: exact for the stored fraction and every 32-bit position, and then rounded by 2^-33 of a turn, where a 32-bit product
// of position and frequency is off by 0.06 at 10^6.  (The fraction itself comes from doubles; what it is off by, 2^-53 of a
// turn at most, the position multiplies.)  The turn's quarter comes from the top bits, and what is left, at most an eighth of a
// turn, goes through sincospi in 32 bits: cosine and sine of the stored angle are off by 2^-23 at most.
//
// Every value is read and written once, so HBM bounds long calls and the launch short ones: 65536 tokens of 32 heads (bf16, d
// = 128, 1.1 GB) take 153 us, 7.0 TB/s, 65536 into the cache (16 q, 2 kv heads, d = 256) 196, 6.8 TB/s; one token 1.8.  Of 8192
// tokens the L2 keeps most of what is written (20.5 us, 134 MB, of them 67 read and 14 to 17 written in HBM; 59% of the issue
// slots): blocks' waves of loads and stores bound them, and of the append (30.4 us, 168 MB) also that every
// store to a page waits for a chain of token, row, table and page.  A block takes a few tokens with all their
// heads: its threads' values are on their way while it looks up the tokens' rows and pages and works out the tokens' cosines
// and sines, which all heads share, in shared memory.  A thread reads and writes both values of a pair, so a call may work
// in place.
#include <algorithm>

#include "gdn_kv.cuh"

namespace gdn {

namespace {

constexpr int kHeld = 4;      // items of a thread whose values are on their way
constexpr int kTokens = 4;    // of a block, at most: a warp looks up each
constexpr int kPairs = 136;   // of a head, with those that fill up the last vector

enum Pairs { kHalf, kHalfAny, kInterleaved };  // kHalfAny: halves that 16-byte vectors do not fit
// Threads of a block: more than items of a head, of which there are up to 32, or 255 where an item is two values.
__host__ __device__ constexpr int threads_of(int pairs) { return pairs == kHalfAny ? 256 : 128; }

struct TurnParams {
  TurnLaunch a;
  int tb;        // tokens of a block
  int heads;     // of a token, all kinds
  int items;     // of a head
  int turning;   // of them (interleaved: of a head's vectors), those that turn
  int at_once;   // heads that a block goes through at a time
  uint32_t head_magic, item_magic;  // 2^32 / heads + 1, 2^32 / items + 1
};

// n / by where magic = 2^32 / by + 1 and n by < 2^32.
__device__ __forceinline__ int divide(int n, int by, uint32_t magic) { return by == 1 ? n : (int)__umulhi((uint32_t)n, magic); }

// Cosine and sine of pair i at a position, times the magnitude.
__device__ __forceinline__ float2 turn_of(const TurnLaunch& p, int pair, int pos) {
  const uint64_t t = load(p.turns + pair) * (uint64_t)(int64_t)pos + 0x80000000u;
  const uint32_t h = (uint32_t)(t >> 32);  // 2^-32 turns
  const uint32_t quarter = (h + 0x20000000u) >> 30;
  float c, s;
  sincospif((float)(int32_t)(h - (quarter << 30)) * 0x1p-31f, &s, &c);
  if (quarter & 1) {
    const float x = c;
    c = -s;
    s = x;
  }
  if (quarter & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(c * p.magnitude, s * p.magnitude);
}

// Where a token's values come from and go to.
struct Place {
  int32_t g;     // global token, -1: nothing of it is written
  int32_t pos;
  int32_t page;  // 0: its keys and values are not written
  int32_t slot;
};

// The row of a local token: the last one that begins at or before it.  32 rows a step; all lanes call together.
__device__ __forceinline__ int row_of(const KvRowsDev& R, int local) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = R.num_seqs;  // among rows [lo, lo + n), the first of which begins at or before the token
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool before = lane == 0 || (lane * step < n && load(R.qsl + at) <= local);
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, before));
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

__device__ __forceinline__ Place place_of(const TurnLaunch& p, int local, int32_t g) {
  const KvDev& C = p.cache;
  Place w{-1, 0, 0, 0};
  KvRow r;
  if (!load_row_of_token(p.rows, C, local, row_of(p.rows, local), r, p.status)) return w;
  w.pos = r.kv - r.len + (local - r.bos);
  w.slot = w.pos & (C.page_size - 1);
  w.page = page_or_null(load(C.table + (int64_t)r.trow * C.max_pages + w.pos / C.page_size), C, p.status);
  if (w.page > 0 && C.refcount && load(C.refcount + w.page) > 1) {
    set_status(p.status, GDN_STATUS_PAGE_SHARED);
    w.page = 0;
  }
  if (g < 0 || g >= p.num_global) {
    set_status(p.status, GDN_STATUS_TOKEN_RANGE);
    return w;
  }
  w.g = g;
  return w;
}

template <typename T>
struct Vec {
  static constexpr int kN = 16 / (int)sizeof(T);
  union {
    uint4 raw;
    T v[16 / sizeof(T)];
  };
  __device__ Vec() : raw(make_uint4(0, 0, 0, 0)) {}
};

// An item is two vectors of a head: the two that some pairs lie in, or two of those that stay, or, interleaved, any two
// with pairs of their own; or it is a pair or a value that stays, where vectors do not fit the halves.  A thread keeps to
// one item of the heads that it takes, and its neighbours take the neighbouring vectors: an item of two vectors side by side
// would leave every 32 bytes to two stores.
template <typename T, int PAIRS, bool APPEND>
__global__ void __launch_bounds__(threads_of(PAIRS), 1024 / threads_of(PAIRS)) turn_kernel(TurnParams P) {
  constexpr int kThreads = threads_of(PAIRS), VE = 16 / (int)sizeof(T);
  constexpr int E = PAIRS == kHalfAny ? 1 : PAIRS == kHalf ? VE : VE / 2;  // pairs of a vector
  __shared__ float2 cs[kTokens][kPairs];
  __shared__ Place places[kTokens];
  const TurnLaunch& p = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int first = blockIdx.x * P.tb, tokens = min(P.tb, p.num_tokens - first);
  const int half = p.rotary / 2, n = P.turning;
  // (token, head) `row` of the block from `row0` on, `at_once` a step, this thread's item of them
  const int row0 = divide(tid, P.items, P.item_magic), i = tid - row0 * P.items;
  const int rows = row0 < P.at_once ? tokens * P.heads : 0;
  const bool turns = i < n;
  const int ia = PAIRS == kInterleaved || turns ? i * (PAIRS == kHalfAny ? 1 : VE) : 2 * half + (i - n) * E;
  const int ib = PAIRS == kInterleaved ? (i + P.items) * VE : turns ? ia + half : ia + (P.items - n) * E;

  const auto source = [&](int t, int head) {
    const int local = first + t;
    const int64_t g = APPEND && p.rows.tok ? load(p.rows.tok + local) : local;
    if (APPEND && (g < 0 || g >= p.num_global)) return static_cast<const T*>(nullptr);
    if (!APPEND || head < p.Hq) return static_cast<const T*>(p.q) + g * p.q_stride + head * p.d;
    head -= p.Hq;
    return head < p.cache.Hkv ? static_cast<const T*>(p.k) + g * p.k_stride + head * p.d
                              : static_cast<const T*>(p.v) + g * p.v_stride + (head - p.cache.Hkv) * p.d;
  };
  const auto target = [&](const Place& at, int head) {
    if (at.g < 0) return static_cast<T*>(nullptr);
    if (!APPEND || head < p.Hq) return static_cast<T*>(p.q_out) + at.g * p.q_out_stride + head * p.d;
    if (at.page == 0) return static_cast<T*>(nullptr);
    const KvDev& C = p.cache;
    head -= p.Hq;
    const bool key = head < C.Hkv;
    T* pool = static_cast<T*>(key ? C.k : C.v) + at.page * C.page_stride;
    return pool + ((key ? head : head - C.Hkv) * C.page_size + at.slot) * p.d;
  };
  const auto turn = [](T& x, T& y, float2 f) {
    const float xf = to_f32(x), yf = to_f32(y);
    x = from_f32<T>(fmaf(xf, f.x, -yf * f.y));
    y = from_f32<T>(fmaf(yf, f.x, xf * f.y));
  };

  for (int from = 0; from == 0 || from < rows; from += kHeld * P.at_once) {
    Vec<T> a[kHeld], b[kHeld];
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int row = from + u * P.at_once + row0;
      if (row >= rows) break;
      const int t = P.tb == 1 ? 0 : divide(row, P.heads, P.head_magic);
      const T* x = source(t, row - t * P.heads);
      if (!x) continue;
      if (PAIRS == kHalfAny) {
        a[u].v[0] = load(x + ia);
        if (turns) b[u].v[0] = load(x + ib);
      } else {
        a[u].raw = load(reinterpret_cast<const uint4*>(x + ia));
        b[u].raw = load(reinterpret_cast<const uint4*>(x + ib));
      }
    }
    if (from == 0) {
      if (APPEND) {
        if (warp < tokens) {
          const int local = first + warp;
          const Place w = place_of(p, local, p.rows.tok ? load(p.rows.tok + local) : local);
          if (lane == 0) places[warp] = w;
        }
      } else if (tid < tokens) {
        places[tid] = Place{first + tid, load(p.positions + first + tid), 0, 0};
      }
      __syncthreads();
      // pair e of item (or vector) i stands at [e n + i]: neighbouring items' pairs are neighbours
      for (int t = 0; t < tokens; ++t)
        for (int pair = tid; pair < half; pair += kThreads) cs[t][pair % E * n + pair / E] = turn_of(p, pair, places[t].pos);
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int row = from + u * P.at_once + row0;
      if (row >= rows) break;
      const int t = P.tb == 1 ? 0 : divide(row, P.heads, P.head_magic), head = row - t * P.heads;
      T* out = target(places[t], head);
      if (!out) continue;
      const bool turned = turns && (!APPEND || head < p.Hq + p.cache.Hkv);
      if (PAIRS == kHalfAny) {
        if (turned) turn(a[u].v[0], b[u].v[0], cs[t][i]);
        out[ia] = a[u].v[0];
        if (turns) out[ib] = b[u].v[0];
        continue;
      }
      if (turned) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (PAIRS == kHalf) {
            turn(a[u].v[e], b[u].v[e], cs[t][e * n + i]);
          } else {
            if (i * E + e < half) turn(a[u].v[2 * e], a[u].v[2 * e + 1], cs[t][e * n + i]);
            if ((i + P.items) * E + e < half) turn(b[u].v[2 * e], b[u].v[2 * e + 1], cs[t][e * n + i + P.items]);
          }
        }
      }
      *reinterpret_cast<uint4*>(out + ia) = a[u].raw;
      *reinterpret_cast<uint4*>(out + ib) = b[u].raw;
    }
  }
}

template <typename T, int PAIRS, bool APPEND>
cudaError_t launch_pairs(const TurnLaunch& a, cudaStream_t s) {
  constexpr int kThreads = threads_of(PAIRS);
  TurnParams P{};
  P.a = a;
  P.heads = a.Hq + (APPEND ? 2 * a.cache.Hkv : 0);
  P.items = PAIRS == kHalfAny ? a.d - a.rotary / 2 : a.d * (int)sizeof(T) / 32;
  const int pairs = PAIRS == kHalfAny ? 1 : (PAIRS == kHalf ? 16 : 8) / (int)sizeof(T);  // of a vector
  P.turning = (a.rotary / 2 + pairs - 1) / pairs;
  P.at_once = kThreads / P.items;
  P.item_magic = (uint32_t)((1ull << 32) / P.items) + 1;
  P.head_magic = (uint32_t)((1ull << 32) / P.heads) + 1;
  // As many tokens as leave the fewest threads without an item (32 heads of d = 128: 2, 20.7 us for 8192 tokens, 22.0 with one a
  // block), fewer where that leaves SMs without a block.
  const int held = kHeld * P.at_once;
  const auto rounds = [&](int tokens) { return (tokens * P.heads + held - 1) / held; };
  P.tb = 1;
  for (int t = 2; t <= kTokens; ++t)
    if ((int64_t)t * P.heads * P.heads < (1ll << 32) && rounds(t) * P.tb < rounds(P.tb) * t) P.tb = t;  // (see divide)
  P.tb = std::max(1, std::min(P.tb, a.num_tokens / (4 * kSms)));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.num_tokens + P.tb - 1) / P.tb);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, turn_kernel<T, PAIRS, APPEND>, P);
}

template <typename T, bool APPEND>
cudaError_t launch_type(const TurnLaunch& a, cudaStream_t s) {
  if (a.layout == GDN_ROPE_INTERLEAVED) return launch_pairs<T, kInterleaved, APPEND>(a, s);
  return a.rotary / 2 * sizeof(T) % 16 == 0 ? launch_pairs<T, kHalf, APPEND>(a, s) : launch_pairs<T, kHalfAny, APPEND>(a, s);
}

}  // namespace

cudaError_t launch_rope(const TurnLaunch& p, gdn_dtype dtype, cudaStream_t s) {
  return dtype == GDN_BF16 ? launch_type<__nv_bfloat16, false>(p, s) : launch_type<float, false>(p, s);
}

cudaError_t launch_kv_append_rope(const TurnLaunch& p, gdn_dtype dtype, cudaStream_t s) {
  return dtype == GDN_BF16 ? launch_type<__nv_bfloat16, true>(p, s) : launch_type<float, true>(p, s);
}

}  // namespace gdn
