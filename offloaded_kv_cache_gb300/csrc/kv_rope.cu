// kv_rope.cu -- rotary positions: rows of q and k turned in place or apart, and the chunk
// append that turns them on the way into the paged cache and keeps the page index.
//
// A pair (a, b) at position t becomes (a cos - b sin, a sin + b cos), angle t * freq.  In
// fp32 t * freq loses the angle's fraction of a turn at far positions (2^20 * 1 is known
// to 2^-4 radians), and fp64 runs at a few percent of fp32's rate here.  So freq / 2 pi is
// taken as a fraction of a turn in units of 2^-64, and the product with t modulo 2^64 is
// the angle's fraction, exact but for t times the last bit of freq.
//
// Each byte is read and written once, and a pair's sine and cosine serve all heads of a
// kv head's group: memory bounds it, for a few tokens the launch and two round trips.
#include <algorithm>
#include <climits>

#include "kv_append.cuh"
#include "kv_launch.h"
#include "kv_q8.cuh"

namespace kvs {
namespace {

#ifndef KVS_ROPE_VECTORS
#define KVS_ROPE_VECTORS 12
#endif

constexpr int kLanes = 16;   // of a vector: two times 4 channels each
constexpr int kGroups = 16;  // half-warps of a block
constexpr int kFlight = 4;   // vectors in flight per half-warp
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
  int lanes;                      // lanes whose channels are turned
  float scale;
  int tile;                       // tokens per block: a page, or 16
  int per_token;                  // half-warps that share a token's vectors, a power of two
  int heads;                      // kv heads of a block
  int blocks, parts;              // tiles per sequence, blocks per tile
  int first_q;                    // vectors of a kv head before its q heads: its key, its value
  int kinds;                      // vectors of a kv head
  Divisor by_blocks, by_parts, by_kinds;
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

// A lane's two pieces of a vector, 4 channels each, as they lie in memory.
template <class T> struct Piece {
  using Word = uint2;
  Word w[2];
};
template <> struct Piece<float> {
  using Word = uint4;
  Word w[2];
};
__device__ __forceinline__ void unpack4(const uint4 &w, float (&x)[4], float) {
  x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
  x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ uint4 pack4(const float (&x)[4], float) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                    __float_as_uint(x[3]));
}
template <class T> __device__ __forceinline__ void unpack4(const uint2 &w, float (&x)[4], T) {
  const float2 a = unpack2(w.x, T{}), b = unpack2(w.y, T{});
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
template <class T> __device__ __forceinline__ uint2 pack4(const float (&x)[4], T) {
  return make_uint2(pack2(x[0], x[1], T{}), pack2(x[2], x[3], T{}));
}

// Turns a lane's four pairs: channel i of both pieces (halves), or neighbours (interleaved).
template <class T, bool kInter>
__device__ __forceinline__ void turn(Piece<T> &p, const float (&c)[4], const float (&s)[4]) {
  float x[4], y[4], u[4], v[4];
  unpack4(p.w[0], x, T{});
  unpack4(p.w[1], y, T{});
  if constexpr (kInter) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u[2 * i] = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
      u[2 * i + 1] = x[2 * i] * s[i] + x[2 * i + 1] * c[i];
      v[2 * i] = y[2 * i] * c[2 + i] - y[2 * i + 1] * s[2 + i];
      v[2 * i + 1] = y[2 * i] * s[2 + i] + y[2 * i + 1] * c[2 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = x[i] * c[i] - y[i] * s[i];
      v[i] = x[i] * s[i] + y[i] * c[i];
    }
  }
  p.w[0] = pack4(u, T{});
  p.w[1] = pack4(v, T{});
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

// Block (sequence, tile of tokens, kv heads), a half-warp a vector.  per_token half-warps share
// a token, whose sines and cosines each has once for all its vectors; of those, kFlight
// are loaded before the first is turned and stored.  A tile is a page where the index is
// kept, so that its keys meet in one block: they are left in shared memory too, and looked
// over there, in totalOrder, at the end.
template <class T, bool kInter>
__global__ void __launch_bounds__(kLanes * kGroups) rope_kernel(const RopeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];  // [token][kv head][128] keys, with an index only
  pdl_wait();
  const int tid = threadIdx.x, l = tid % kLanes, grp = tid / kLanes;
  const int seq_tile = a.by_parts(blockIdx.x), part = (int)blockIdx.x - seq_tile * a.parts;
  const int b = a.by_blocks(seq_tile), j = seq_tile - b * a.blocks;
  const bool turns = l < a.lanes;
  double freq[4];
  if (turns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) freq[i] = a.freq[4 * l + i];
  }
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
  const int c0 = turns && !kInter ? 4 * l : 8 * l;
  const int c1 = turns && !kInter ? 4 * (a.lanes + l) : 8 * l + 4;
  uint64_t f[4] = {0, 0, 0, 0};
  if (turns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = turns_of(freq[i]);
  }
  using Word = typename Piece<T>::Word;
  const int h0 = part * a.heads, heads = min(a.heads, a.Hkv - h0);
  const int vectors = heads * a.kinds;
  const int sub = grp & (a.per_token - 1);
  for (int i = lo + grp / a.per_token; i < hi; i += kGroups / a.per_token) {
    const long long row = r.q0 + i;
    const int pos = a.at ? a.at[row] : r.len + i;
    float c[4], s[4];
    for (int v0 = sub; v0 < vectors; v0 += kFlight * a.per_token) {
      Piece<T> x[kFlight];
      T *dst[kFlight];
      int kind[kFlight], head[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int v = v0 + k * a.per_token;
        dst[k] = nullptr;
        if (v >= vectors) continue;
        head[k] = a.by_kinds(v);
        kind[k] = v - head[k] * a.kinds;
        const int h = h0 + head[k];
        const T *src;
        if (kind[k] < a.first_q) {
          // (without keys, the first vector would be the value: there is no such call)
          src = static_cast<const T *>(kind[k] ? a.v : a.k) + (row * a.Hkv + h) * kHeadDim;
          // (rows of the cache fit int32)
          const long long to =
              a.bt ? ((long long)ph * a.Hkv + h) * a.ps + slot0 + (i - lo) : row * a.Hkv + h;
          if (a.bt && ph < 0) continue;
          dst[k] = static_cast<T *>(kind[k] ? a.v_out : a.k_out) + to * kHeadDim;
        } else {
          const long long at = row * a.Hq + (long long)h * a.G + kind[k] - a.first_q;
          src = static_cast<const T *>(a.q) + at * kHeadDim;
          dst[k] = static_cast<T *>(a.q_out) + at * kHeadDim;
        }
        x[k].w[0] = *reinterpret_cast<const Word *>(src + c0);
        x[k].w[1] = *reinterpret_cast<const Word *>(src + c1);
      }
      if (v0 == sub && turns) {  // (while the first vectors are on their way)
#pragma unroll
        for (int k = 0; k < 4; ++k) cos_sin(f[k], pos, a.scale, c[k], s[k]);
      }
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        if (!dst[k]) continue;
        if (turns && !(kind[k] == 1 && a.first_q == 2)) turn<T, kInter>(x[k], c, s);
        *reinterpret_cast<Word *>(dst[k] + c0) = x[k].w[0];
        *reinterpret_cast<Word *>(dst[k] + c1) = x[k].w[1];
        if (a.mm && kind[k] == 0) {
          T *keep = reinterpret_cast<T *>(smem) + ((i - lo) * heads + head[k]) * kHeadDim;
          *reinterpret_cast<Word *>(keep + c0) = x[k].w[0];
          *reinterpret_cast<Word *>(keep + c1) = x[k].w[1];
        }
      }
    }
  }
  if (!a.mm || ph < 0) return;
  __syncthreads();
  constexpr int kWords = kHeadDim * sizeof(T) / 4;
  for (int i = tid; i < heads * kWords; i += kLanes * kGroups) {
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
  if (smem > 48 * 1024) {
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
    a.lanes = rope->rotary_dim / 8;
    a.scale = rope->scale;
  }
  a.tile = mm ? a.ps : 16;
  if (!rope_grid(s, c, bt != nullptr, a.tile, &a.blocks)) return cudaErrorInvalidConfiguration;
  a.per_token = 1;
  const int tokens = std::min({c->max_q_len, c->total_q, a.tile});
  while (2 * a.per_token * tokens <= kGroups) a.per_token *= 2;
  a.first_q = (k ? 1 : 0) + (v ? 1 : 0);
  a.kinds = a.first_q + (q ? a.G : 0);
  a.by_kinds = Divisor::of(a.kinds);
  // kv heads of a block: a dozen vectors a half-warp, or as many half-warps as vectors; no
  // more than whose keys the shared memory takes (a page of 128 tokens in fp32 is 64 KB)
  a.heads = std::max(1, (a.per_token > 1 ? a.per_token : KVS_ROPE_VECTORS) / a.kinds);
  const int key_bytes = tokens * kHeadDim * (s->dtype == KV_F32 ? 4 : 2);  // of a kv head's
  if (ctx_out && ctx_out == ctx && a.blocks == 1)
    a.heads = a.Hkv;  // one block per sequence: it can write the lengths that it alone reads
  if (mm) a.heads = std::min(a.heads, kKeyBytes / key_bytes);
  a.heads = std::min(a.heads, a.Hkv);
  a.parts = (a.Hkv + a.heads - 1) / a.heads;
  a.by_blocks = Divisor::of(a.blocks);
  a.by_parts = Divisor::of(a.parts);
  const bool later = ctx_out && ctx_out == ctx && (a.blocks > 1 || a.parts > 1);
  a.write_lens = ctx_out && !later;
  const dim3 grid((unsigned)(a.blocks * s->batch * a.parts)), block(kLanes * kGroups);
  const size_t smem = mm ? (size_t)a.heads * key_bytes : 0;
  const bool inter = rope && rope->interleaved;
  cudaError_t e;
  switch (s->dtype) {
    case KV_F32:
      e = inter ? rope_go(rope_kernel<float, true>, grid, block, smem, st, a)
                : rope_go(rope_kernel<float, false>, grid, block, smem, st, a);
      break;
    case KV_F16:
      e = inter ? rope_go(rope_kernel<__half, true>, grid, block, smem, st, a)
                : rope_go(rope_kernel<__half, false>, grid, block, smem, st, a);
      break;
    default:
      e = inter ? rope_go(rope_kernel<__nv_bfloat16, true>, grid, block, smem, st, a)
                : rope_go(rope_kernel<__nv_bfloat16, false>, grid, block, smem, st, a);
  }
  if (e == cudaSuccess && later)
    e = launch_pdl(advance_kernel<RopeArgs>, dim3(s->batch), dim3(256), 0, st, a);
  return e;
}

}  // namespace kvs
