// kv_rope.cu -- rotary positions: rows of q and k turned in place or apart, and the chunk
// append that turns them on the way into the paged cache and keeps the page index.
//
// A pair (a, b) at position t becomes (a cos - b sin, a sin + b cos), angle t * freq.  In
// fp32 t * freq loses the angle's fraction of a turn at far positions (2^20 * 1 is known
// to 2^-4 radians), and fp64 runs at a few percent of fp32's rate here.  So freq / 2 pi is
// taken as a fraction of a turn in units of 2^-64, rounded down, and its product with t modulo
// 2^64 is the angle's fraction.  It is off by t times what freq / 2 pi is: 2^-64 for the unit,
// freq * 2^-66 for 1 / 2 pi's last bit; and 2^-33 for the 32 bits that sine and cosine take.
//
// Each byte is read and written once, and a pair's sine and cosine serve all heads of a
// kv head's group: memory bounds it, for a few tokens the launch and two round trips.
// 32 prompts of <= 513 tokens, 32/32 heads, f16: 40 us, 230 MB, 5.8 TB/s; append of 4 x <= 2048,
// 32/8 heads, bf16, with the index: 20 us, 102 MB, 5.2 TB/s; 32 x 1: 2.4 us, append 3.1.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "kv_append.cuh"
#include "kv_launch.h"
#include "kv_q8.cuh"

namespace kvs {
namespace {

#ifndef KVS_ROPE_VECTORS
#define KVS_ROPE_VECTORS 24
#endif
#ifndef KVS_ROPE_FILL
#define KVS_ROPE_FILL (152 * 1024 * 3 / 2)  // threads
#endif
#ifndef KVS_ROPE_FLIGHT
#define KVS_ROPE_FLIGHT 16  // pairs of a lane in flight (32: the prompts above 45 us)
#endif

constexpr int kThreads = 256;   // or twice as many, for pages of more than 16 tokens
constexpr int kMaxAtOnce = 32;  // tokens
constexpr int kPairs = kHeadDim / 2;
constexpr int kKeyBytes = 64 * 1024;  // of keys that a block keeps for the index

struct RopeArgs {
  const void *q, *k, *v;          // rows; null: left out
  void *q_out, *k_out, *v_out;    // k, v: rows, or the cache's pages
  void *mm;                       // the page index, or null
  const double *freq;             // null: nothing is turned
  const int32_t *at;              // positions, or null
  const int32_t *q_start, *bt, *ctx;
  int32_t *ctx_out;
  int *status;
  long long nphys;
  int Hq, Hkv, G, ps, ps_log2, maxP, total_q, max_q_len;
  int pairs;                      // that are turned
  float scale;
  int tile;                       // tokens per block: a page, or 16
  int per_token;                  // groups that share a token's vectors, a power of two
  int heads;                      // kv heads of a block
  int blocks, parts;              // tiles per sequence, blocks per tile
  Divisor by_blocks, by_parts;
  int write_lens;
};

// freq / 2 pi modulo 1 in units of 2^-64: freq = m * 2^(x - 52), 1 / 2 pi = A * 2^-66
// with A < 2^64, so the fraction is (m * A) >> (54 - x).  (x <= 53)
__device__ __forceinline__ uint64_t turns_of(double freq) {
  const uint64_t u = (uint64_t)__double_as_longlong(freq);
  const int x = (int)((u >> 52) & 0x7FF) - 1023, s = 54 - x;
  const uint64_t m = (u & 0xFFFFFFFFFFFFFull) | (1ull << 52), A = 0xA2F9836E4E44152Aull;
  const uint64_t lo = m * A, hi = __umul64hi(m, A);
  uint64_t f = 0;  // (a frequency below 2^-64 turns nothing)
  if (s >= 64 && s < 128) f = hi >> (s - 64);
  if (s > 0 && s < 64) f = (lo >> s) | (hi << (64 - s));
  return (u >> 63) ? 0ull - f : f;
}
// (others, infinities and NaN among them, give 0 above: they turn nothing)
__device__ __forceinline__ bool turnable(double freq) {
  return ((uint64_t)__double_as_longlong(freq) >> 52 & 0x7FF) < 1023 + 54;
}
// cosine and sine of f * pos turns: the nearest quarter and the rest, within an eighth
__device__ __forceinline__ void cos_sin(uint64_t f, int pos, float scale, float &c, float &s) {
  const uint64_t a = f * (uint64_t)(long long)pos;
  const uint32_t turn = (uint32_t)((a + 0x80000000ull) >> 32);
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  float c0, s0;
  sincospif((float)(int32_t)(turn - (quarter << 30)) * 0x1p-31f, &s0, &c0);
  const float u = quarter & 1 ? s0 : c0, v = quarter & 1 ? c0 : s0;
  c = (((quarter + 1) & 2) ? -u : u) * scale;
  s = ((quarter & 2) ? -v : v) * scale;
}

// A lane's two pieces of a vector, kCh channels each, as they lie in memory: 16 bytes, or, of 16-bit
// data whose turned pairs are an odd number of fours, 8 (16 x <= 2000 tokens, 32/8 heads, bf16:
// 48.3 us with 16 bytes, 53.4 with 8).
template <class T, int kCh> struct Piece {
  static constexpr int kWords = kCh * (int)sizeof(T) / 4;
  using Word = std::conditional_t<kWords == 4, uint4, uint2>;
  alignas(16) uint32_t w[2][kWords];
  __device__ __forceinline__ void load(int i, const T *src) {
    *reinterpret_cast<Word *>(w[i]) = *reinterpret_cast<const Word *>(src);
  }
  __device__ __forceinline__ void store(int i, T *dst) const {
    *reinterpret_cast<Word *>(dst) = *reinterpret_cast<const Word *>(w[i]);
  }
};
template <int kCh>
__device__ __forceinline__ void unpack(const uint32_t (&w)[kCh], float (&x)[kCh], float) {
#pragma unroll
  for (int i = 0; i < kCh; ++i) x[i] = __uint_as_float(w[i]);
}
template <int kCh>
__device__ __forceinline__ void pack(const float (&x)[kCh], uint32_t (&w)[kCh], float) {
#pragma unroll
  for (int i = 0; i < kCh; ++i) w[i] = __float_as_uint(x[i]);
}
template <class T, int kCh>
__device__ __forceinline__ void unpack(const uint32_t (&w)[kCh / 2], float (&x)[kCh], T) {
#pragma unroll
  for (int i = 0; i < kCh / 2; ++i) {
    const float2 a = unpack2(w[i], T{});
    x[2 * i] = a.x;
    x[2 * i + 1] = a.y;
  }
}
template <class T, int kCh>
__device__ __forceinline__ void pack(const float (&x)[kCh], uint32_t (&w)[kCh / 2], T) {
#pragma unroll
  for (int i = 0; i < kCh / 2; ++i) w[i] = pack2(x[2 * i], x[2 * i + 1], T{});
}

// Turns a lane's pairs: channel i of both pieces (halves), or neighbours (interleaved).
template <class T, int kCh, bool kInter>
__device__ __forceinline__ void turn(Piece<T, kCh> &p, const float (&c)[kCh], const float (&s)[kCh]) {
  float x[kCh], y[kCh], u[kCh], v[kCh];
  unpack(p.w[0], x, T{});
  unpack(p.w[1], y, T{});
  if constexpr (kInter) {
#pragma unroll
    for (int i = 0; i < kCh / 2; ++i) {
      const int k = kCh / 2 + i;
      u[2 * i] = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
      u[2 * i + 1] = x[2 * i] * s[i] + x[2 * i + 1] * c[i];
      v[2 * i] = y[2 * i] * c[k] - y[2 * i + 1] * s[k];
      v[2 * i + 1] = y[2 * i] * s[k] + y[2 * i + 1] * c[k];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      u[i] = x[i] * c[i] - y[i] * s[i];
      v[i] = x[i] * s[i] + y[i] * c[i];
    }
  }
  pack(u, p.w[0], T{});
  pack(v, p.w[1], T{});
}

// The minimum and maximum of one word of the keys of `count` tokens, `stride` words apart, and
// of what the index held: two channels of 16 bits, or one of 32.
template <class T>
__device__ __forceinline__ void word_bounds(const uint32_t *at, int stride, int count, bool old,
                                            uint32_t *lo, uint32_t *hi) {
  if constexpr (sizeof(T) == 2) {
    uint32_t mn = old ? key16x2(*lo) : ~0u, mx = old ? key16x2(*hi) : 0;
#pragma unroll 4
    for (int i = 0; i < count; ++i) {
      const uint32_t key = key16x2(at[i * stride]);
      mn = __vminu2(mn, key);
      mx = __vmaxu2(mx, key);
    }
    *lo = unkey16x2(mn);
    *hi = unkey16x2(mx);
  } else {
    uint32_t mn = old ? key32(*lo) : ~0u, mx = old ? key32(*hi) : 0;
#pragma unroll 4
    for (int i = 0; i < count; ++i) {
      const uint32_t key = key32(at[i * stride]);
      mn = min(mn, key);
      mx = max(mx, key);
    }
    *lo = unkey32(mn);
    *hi = unkey32(mx);
  }
}

// Block (sequence, tile of tokens, kv heads), 16 or 32 tokens of the tile at a time: first a
// thread a pair takes the tokens' sines and cosines into shared memory, then a group of 8 or 16
// lanes a vector turns and stores, kFlight vectors loaded before the first is stored, the first of
// them before the angles are taken (after: the prompts above 41 us, the append 20.4); per_token
// groups share a token.  A tile is a page where the index is kept, so that its keys meet
// in one block: they are left in shared memory too, and looked over there, in totalOrder, at
// the end.
template <class T, int kCh, bool kInter>
__global__ void __launch_bounds__(2 * kThreads, sizeof(T) == 2 ? 2 : 1) rope_kernel(const RopeArgs a) {
  constexpr int kLanes = kHeadDim / 2 / kCh, kFlight = KVS_ROPE_FLIGHT / kCh;
  extern __shared__ __align__(16) uint8_t smem[];  // [token][kv head][128] keys, with an index only
  __shared__ __align__(16) float cosine[kMaxAtOnce][kPairs], sine[kMaxAtOnce][kPairs];
  pdl_wait();
  const int tid = threadIdx.x, l = tid % kLanes, grp = tid / kLanes;
  const int groups = blockDim.x / kLanes, at_once = groups / a.per_token;  // tokens at a time
  const int seq_tile = a.by_parts(blockIdx.x), part = (int)blockIdx.x - seq_tile * a.parts;
  const int b = a.by_blocks(seq_tile), j = seq_tile - b * a.blocks;
  const int lanes = a.pairs / kCh;  // that turn
  const bool turns = l < lanes;
  const int pair = tid % kPairs;
  double freq = 0.0;
  if (pair < a.pairs) freq = a.freq[pair];
  RowSpan r{a.q_start[b], a.q_start[b + 1] - a.q_start[b], 0};
  if (a.bt) {
    r = append_span(a, b);
  } else {
    if (a.ctx) r.len = a.ctx[b];
    if (r.q0 < 0 || r.n < 0 || (long long)r.q0 + r.n > a.total_q || r.n > a.max_q_len || r.len < 0 ||
        (long long)r.len + r.n > INT_MAX)
      r.n = -1;
  }
  if (j == 0 && part == 0) {
    const bool ok = r.n >= 0 && (!a.bt || pages_ok(a, b, r));  // ends in a barrier when it asks
    if (tid == 0) {
      if (!ok) flag_error(a.status, KV_ERR_BOUNDS);
      if (a.write_lens) a.ctx_out[b] = ok ? r.len + r.n : r.len;
    }
    if (tid < kPairs && !turnable(freq)) flag_error(a.status, KV_ERR_BOUNDS);
  }
  pdl_trigger();
  // the block's tokens, counted from the chunk's start
  const int skew = a.bt ? r.len & (a.tile - 1) : 0;
  const long long t0 = (long long)j * a.tile - skew;
  const int lo = (int)max(t0, 0ll), hi = (int)min(t0 + a.tile, (long long)r.n);
  if (lo >= hi) return;
  int ph = -1, slot0 = 0;
  if (a.bt) {
    ph = a.bt[(long long)b * a.maxP + ((r.len + lo) >> a.ps_log2)];
    if (ph < 0 || ph >= a.nphys) ph = -1;  // recorded by the sequence's first block
    slot0 = (r.len + lo) & (a.ps - 1);
  }
  const int c0 = turns && !kInter ? kCh * l : 2 * kCh * l;
  const int c1 = turns && !kInter ? kCh * (lanes + l) : 2 * kCh * l + kCh;
  const int h0 = part * a.heads, heads = min(a.heads, a.Hkv - h0), sub = grp & (a.per_token - 1);
  // A token's vectors: its keys, its values, q heads; K's and V's heads lie a page's tokens
  // apart in the cache.
  const int keys = a.k ? heads : 0, rows_kv = keys + (a.v ? heads : 0);
  const int count = rows_kv + (a.q ? heads * a.G : 0), apart = a.bt ? a.ps * kHeadDim : kHeadDim;
  const uint64_t f = turns_of(freq);
  for (int i0 = lo; i0 < hi; i0 += at_once) {
    const int tokens = min(at_once, hi - i0);
    const int mine = grp / a.per_token, i = i0 + mine;
    const long long row = r.q0 + i;
    const long long in = (row * a.Hkv + h0) * kHeadDim;
    const long long at = (row * a.Hq + (long long)h0 * a.G) * kHeadDim;
    Piece<T, kCh> x[kFlight];
    const auto load = [&](int v0) {
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int v = v0 + k * a.per_token;
        if (v >= count) continue;
        const T *src = v < keys      ? static_cast<const T *>(a.k) + in + v * kHeadDim
                       : v < rows_kv ? static_cast<const T *>(a.v) + in + (v - keys) * kHeadDim
                                     : static_cast<const T *>(a.q) + at + (v - rows_kv) * kHeadDim;
        x[k].load(0, src + c0);
        x[k].load(1, src + c1);
      }
    };
    if (mine < tokens) load(sub);
    if (pair < a.pairs) {
      for (int k = tid / kPairs; k < tokens; k += blockDim.x / kPairs)
        cos_sin(f, a.at ? a.at[r.q0 + i0 + k] : r.len + i0 + k, a.scale, cosine[k][pair], sine[k][pair]);
    }
    __syncthreads();
    if (mine < tokens) {
      // (rows of the cache fit int32)
      const long long out =
          a.bt ? (((long long)ph * a.Hkv + h0) * a.ps + slot0 + (i - lo)) * kHeadDim : in;
      const bool there = !a.bt || ph >= 0;
      float c[kCh], s[kCh];
      if (turns) {
#pragma unroll
        for (int k = 0; k < kCh; k += 4) {
          const float4 u = *reinterpret_cast<const float4 *>(&cosine[mine][kCh * l + k]);
          const float4 v = *reinterpret_cast<const float4 *>(&sine[mine][kCh * l + k]);
          c[k] = u.x; c[k + 1] = u.y; c[k + 2] = u.z; c[k + 3] = u.w;
          s[k] = v.x; s[k + 1] = v.y; s[k + 2] = v.z; s[k + 3] = v.w;
        }
      }
#pragma unroll 1
      for (int v0 = sub; v0 < count;) {
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
          const int v = v0 + k * a.per_token;
          if (v >= count || (v < rows_kv && !there)) continue;
          T *dst = v < keys      ? static_cast<T *>(a.k_out) + out + (long long)v * apart
                   : v < rows_kv ? static_cast<T *>(a.v_out) + out + (long long)(v - keys) * apart
                                 : static_cast<T *>(a.q_out) + at + (v - rows_kv) * kHeadDim;
          if (turns && (v < keys || v >= rows_kv)) turn<T, kCh, kInter>(x[k], c, s);
          x[k].store(0, dst + c0);
          x[k].store(1, dst + c1);
          if (a.mm && v < keys) {
            T *keep = reinterpret_cast<T *>(smem) + ((i - lo) * heads + v) * kHeadDim;
            x[k].store(0, keep + c0);
            x[k].store(1, keep + c1);
          }
        }
        v0 += kFlight * a.per_token;
        if (v0 < count) load(v0);
      }
    }
    __syncthreads();
  }
  if (!a.mm || ph < 0) return;
  constexpr int kWords = kHeadDim * sizeof(T) / 4;
  for (int i = tid; i < heads * kWords; i += blockDim.x) {
    const int h = i / kWords, w = i % kWords;
    uint32_t *e = static_cast<uint32_t *>(a.mm) + (((long long)ph * a.Hkv + h0 + h) * 2) * kWords + w;
    uint32_t mn = 0, mx = 0;
    if (slot0 > 0) mn = e[0], mx = e[kWords];
    word_bounds<T>(reinterpret_cast<const uint32_t *>(smem) + i, heads * kWords, hi - lo, slot0 > 0,
                   &mn, &mx);
    e[0] = mn;
    e[kWords] = mx;
  }
}

template <class K>
cudaError_t rope_go(K kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                    const RopeArgs &a) {
  if (smem > 16 * 1024) {  // (beside the angles)
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyBytes);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, grid, block, smem, st, a);
}

}  // namespace

// The launch's blocks, which have to count in int32.
bool rope_grid(const kv_shape *s, const kv_chunk *c, bool paged, int tile, int *blocks) {
  const long long n = std::min(c->max_q_len, c->total_q);
  // (a chunk that starts inside a tile touches one more)
  const long long k = paged ? (n + tile - 2) / tile + 1 : (n + tile - 1) / tile;
  *blocks = (int)k;
  return k * s->batch * s->num_kv_heads <= INT_MAX;
}

cudaError_t launch_rope(const kv_shape *s, const kv_chunk *c, const kv_rope_plan *rope,
                        const void *q, void *q_out, const void *k, void *k_out, const void *v,
                        void *v_out, const int32_t *bt, const int32_t *ctx, int32_t *ctx_out,
                        void *mm, int *status, cudaStream_t st) {
  RopeArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.k_out = k_out;
  a.v_out = v_out;
  a.mm = mm;
  a.q_start = c->q_start;
  a.bt = bt;
  a.ctx = ctx;
  a.ctx_out = ctx_out;
  a.status = status;
  a.nphys = s->num_phys_pages;
  a.Hq = s->num_q_heads;
  a.Hkv = s->num_kv_heads;
  a.G = a.Hq / a.Hkv;
  a.ps = s->page_size;
  a.ps_log2 = __builtin_ctz(a.ps);
  a.maxP = s->max_pages_per_seq;
  a.total_q = c->total_q;
  a.max_q_len = c->max_q_len;
  a.scale = 1.f;
  if (rope) {
    a.freq = rope->freq;
    a.at = rope->positions;
    a.pairs = rope->rotary_dim / 2;
    a.scale = rope->scale;
  }
  a.tile = mm ? a.ps : 16;
  if (!rope_grid(s, c, bt != nullptr, a.tile, &a.blocks)) return cudaErrorInvalidConfiguration;
  const int tokens = std::min({c->max_q_len, c->total_q, a.tile});
  const int threads = tokens > 16 ? 2 * kThreads : kThreads;
  const bool wide = s->dtype != KV_F32 && a.pairs % 8 == 0;
  const int groups = threads / (kHeadDim / 2 / (wide ? 8 : 4));
  a.per_token = 1;
  while (2 * a.per_token * tokens <= groups || a.per_token * kMaxAtOnce < groups) a.per_token *= 2;
  const int kinds = (k ? 1 : 0) + (v ? 1 : 0) + (q ? a.G : 0);
  const int row_bytes = kHeadDim * (s->dtype == KV_F32 ? 4 : 2), key_bytes = tokens * row_bytes;
  // kv heads of a block: up to KVS_ROPE_VECTORS of a token's vectors, which share its angles, but
  // blocks enough to fill the GPU one and a half times; of a few tokens, as many groups as vectors
  // and a thread for a word of the index; no more than whose keys the shared memory takes (a page
  // of 128 tokens in fp32 is 64 KB).  Append, us:
  //   4 x 2048 tokens, 32/8 heads, bf16: pages of 16, 2 / 4 / 8 heads 22.2 / 20.6 / 25.2; of 64,
  //     1 / 2 / 4 heads 28.7 / 22.2 / 30.6; of 128, 1 / 2 heads 27.8 / 35.5; fp32, pages of 16,
  //     2 / 4 / 8 heads 38.9 / 37.0 / 36.1
  //   16 x 2000, 64/8 heads, f16, pages of 64: 1 / 2 heads 114 / 99; 1 x 513, 32/8: 10.4 / 13.1
  //   256 x 1, 32/8 heads, f16: 2 / 4 / 5 heads 6.9 / 4.7 / 5.4
  if (tokens <= 8) {
    a.heads = a.per_token / kinds;
    if (mm) a.heads = std::min(a.heads, threads * 4 / row_bytes);
  } else {
    a.heads = std::min(KVS_ROPE_VECTORS / kinds, a.Hkv);
    while (a.heads > 1 &&
           (long long)a.blocks * s->batch * ((a.Hkv + a.heads - 1) / a.heads) * threads < KVS_ROPE_FILL)
      --a.heads;
  }
  a.heads = std::max(1, a.heads);
  if (ctx_out && ctx_out == ctx && a.blocks == 1)
    a.heads = a.Hkv;  // one block per sequence: it can write the lengths that it alone reads
  if (mm) a.heads = std::min(a.heads, kKeyBytes / key_bytes);
  a.heads = std::min(a.heads, a.Hkv);
  a.parts = (a.Hkv + a.heads - 1) / a.heads;
  a.by_blocks = Divisor::of(a.blocks);
  a.by_parts = Divisor::of(a.parts);
  const bool later = ctx_out && ctx_out == ctx && (a.blocks > 1 || a.parts > 1);
  a.write_lens = ctx_out && !later;
  const dim3 grid((unsigned)(a.blocks * s->batch * a.parts)), block(threads);
  const size_t smem = mm ? (size_t)a.heads * key_bytes : 0;
  const bool inter = rope && rope->interleaved;
  const auto go = [&](auto t) {
    using T = decltype(t);
    constexpr int kCh = 16 / sizeof(T);
    if constexpr (kCh == 8) {
      if (!wide)
        return inter ? rope_go(rope_kernel<T, 4, true>, grid, block, smem, st, a)
                     : rope_go(rope_kernel<T, 4, false>, grid, block, smem, st, a);
    }
    return inter ? rope_go(rope_kernel<T, kCh, true>, grid, block, smem, st, a)
                 : rope_go(rope_kernel<T, kCh, false>, grid, block, smem, st, a);
  };
  cudaError_t e = s->dtype == KV_F32   ? go(float{})
                  : s->dtype == KV_F16 ? go(__half{})
                                       : go(__nv_bfloat16{});
  if (e == cudaSuccess && later)
    e = launch_pdl(advance_kernel<RopeArgs>, dim3(s->batch), dim3(256), 0, st, a);
  return e;
}

}  // namespace kvs
