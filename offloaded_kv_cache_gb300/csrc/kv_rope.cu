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

constexpr int kLanes = 16;        // of a vector: two times 4 channels each
constexpr int kGroups = 16;       // half-warps per kv head of a block
constexpr int kHeads = 4;         // q vectors in flight per half-warp

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
  int heads;                      // kv heads a block walks
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

// Block (sequence, tile of tokens, kv heads): blockDim.x / 256 kv heads at a time, 16
// half-warps each.  per_token half-warps share a token: its key (the first one), value
// and the group's q heads.  A tile is a page where the index is kept, so that its keys
// meet in one block, whose minima and maxima are taken over totalOrder keys in shared
// memory, in any order.
template <class T, bool kInter>
__global__ void __launch_bounds__(512) rope_kernel(const RopeArgs a) {
  extern __shared__ uint32_t bounds[];  // [kv heads at a time][2][128], with an index only
  pdl_wait();
  const int tid = threadIdx.x, l = tid % kLanes;
  const int seq_tile = a.by_parts(blockIdx.x), part = (int)blockIdx.x - seq_tile * a.parts;
  const int b = a.by_blocks(seq_tile), j = seq_tile - b * a.blocks;
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
  const bool turns = l < a.lanes;
  const int c0 = turns && !kInter ? 4 * l : 8 * l;
  const int c1 = turns && !kInter ? 4 * (a.lanes + l) : 8 * l + 4;
  uint64_t f[4] = {0, 0, 0, 0};
  if (turns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = turns_of(a.freq[4 * l + i]);
  }
  using Word = typename Piece<T>::Word;
  auto load = [&](const void *base, long long vec) {
    const T *p = static_cast<const T *>(base) + vec * kHeadDim;
    Piece<T> x;
    x.w[0] = *reinterpret_cast<const Word *>(p + c0);
    x.w[1] = *reinterpret_cast<const Word *>(p + c1);
    return x;
  };
  auto store = [&](void *base, long long vec, const Piece<T> &x) {
    T *p = static_cast<T *>(base) + vec * kHeadDim;
    *reinterpret_cast<Word *>(p + c0) = x.w[0];
    *reinterpret_cast<Word *>(p + c1) = x.w[1];
  };
  const int at_once = blockDim.x / (kLanes * kGroups), mine = tid / (kLanes * kGroups);
  const int grp = tid / kLanes % kGroups, sub = grp & (a.per_token - 1);
  const int first = grp / a.per_token, step = kGroups / a.per_token;
  const int h_end = min(a.Hkv, (part + 1) * a.heads);
  for (int h0 = part * a.heads; h0 < h_end; h0 += at_once) {
    const int h = h0 + mine;
    const bool on = h < h_end;
    uint32_t *low = bounds + mine * 2 * kHeadDim, *high = low + kHeadDim;
    if (a.mm) {
      __syncthreads();
      for (int i = tid % (kLanes * kGroups); i < kHeadDim; i += kLanes * kGroups) {
        low[i] = ~0u;
        high[i] = 0;
      }
      __syncthreads();
    }
    uint32_t mn[8], mx[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mn[i] = ~0u;
      mx[i] = 0;
    }
    bool any = false;
    for (int i = lo + first; on && i < hi; i += step) {
      const long long row = r.q0 + i;
      float c[4], s[4];
      const int pos = a.at ? a.at[row] : r.len + i;
      // (rows of the cache fit int32)
      const long long to =
          a.bt ? ((long long)ph * a.Hkv + h) * a.ps + slot0 + (i - lo) : row * a.Hkv + h;
      const bool has = !a.bt || ph >= 0;
      if (turns) {
#pragma unroll
        for (int k = 0; k < 4; ++k) cos_sin(f[k], pos, a.scale, c[k], s[k]);
      }
      // vectors of the token: 0 its key, 1 its value, 2 .. the q heads
      if (a.k && sub == 0 && has) {
        Piece<T> x = load(a.k, row * a.Hkv + h);
        if (turns) turn<T, kInter>(x, c, s);
        store(a.k_out, to, x);
        if (a.mm) {
          float y[4];
          any = true;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            unpack4(x.w[w], y, T{});
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t key = key32(__float_as_uint(y[k]));
              mn[4 * w + k] = min(mn[4 * w + k], key);
              mx[4 * w + k] = max(mx[4 * w + k], key);
            }
          }
        }
      }
      if (a.v && sub == (1 & (a.per_token - 1)) && has)
        store(a.v_out, to, load(a.v, row * a.Hkv + h));
      if (a.q) {
        const long long q0 = row * a.Hq + (long long)h * a.G;
        for (int g = (sub - 2) & (a.per_token - 1); g < a.G; g += kHeads * a.per_token) {
          Piece<T> x[kHeads];
#pragma unroll
          for (int k = 0; k < kHeads; ++k)
            if (g + k * a.per_token < a.G) x[k] = load(a.q, q0 + g + k * a.per_token);
#pragma unroll
          for (int k = 0; k < kHeads; ++k)
            if (g + k * a.per_token < a.G) {
              if (turns) turn<T, kInter>(x[k], c, s);
              store(a.q_out, q0 + g + k * a.per_token, x[k]);
            }
        }
      }
    }
    if (!a.mm) continue;
    if (any) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          atomicMin(&low[(w ? c1 : c0) + k], mn[4 * w + k]);
          atomicMax(&high[(w ? c1 : c0) + k], mx[4 * w + k]);
        }
    }
    __syncthreads();
    if (on && ph >= 0 && grp < 2) {
      // a half-warp writes the minima, another one the maxima, eight channels a lane
      T *e = static_cast<T *>(a.mm) + (((long long)ph * a.Hkv + h) * 2 + grp) * kHeadDim + 8 * l;
      const uint32_t *from = (grp ? high : low) + 8 * l;
      float old[8], x[8];
      if (slot0 > 0) load8(e, old);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint32_t key = from[k];
        if (slot0 > 0) {
          const uint32_t was = key32(__float_as_uint(old[k]));
          key = grp ? max(key, was) : min(key, was);
        }
        x[k] = __uint_as_float(unkey32(key));
      }
      store8(e, x);
    }
  }
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
  a.heads = 1;
  int at_once = 1;
  if (ctx_out && ctx_out == ctx && a.blocks == 1) {
    // one block per sequence: it can write the lengths that it alone reads
    a.heads = a.Hkv;
    at_once = std::min(2, a.Hkv);
  }
  a.parts = (a.Hkv + a.heads - 1) / a.heads;
  a.by_blocks = Divisor::of(a.blocks);
  a.by_parts = Divisor::of(a.parts);
  const bool later = ctx_out && ctx_out == ctx && (a.blocks > 1 || a.parts > 1);
  a.write_lens = ctx_out && !later;
  const dim3 grid((unsigned)(a.blocks * s->batch * a.parts)), block(kLanes * kGroups * at_once);
  const size_t smem = mm ? (size_t)at_once * 2 * kHeadDim * 4 : 0;
  const bool inter = rope && rope->interleaved;
  cudaError_t e;
  switch (s->dtype) {
    case KV_F32:
      e = inter ? launch_pdl(rope_kernel<float, true>, grid, block, smem, st, a)
                : launch_pdl(rope_kernel<float, false>, grid, block, smem, st, a);
      break;
    case KV_F16:
      e = inter ? launch_pdl(rope_kernel<__half, true>, grid, block, smem, st, a)
                : launch_pdl(rope_kernel<__half, false>, grid, block, smem, st, a);
      break;
    default:
      e = inter ? launch_pdl(rope_kernel<__nv_bfloat16, true>, grid, block, smem, st, a)
                : launch_pdl(rope_kernel<__nv_bfloat16, false>, grid, block, smem, st, a);
  }
  if (e == cudaSuccess && later)
    e = launch_pdl(advance_kernel<RopeArgs>, dim3(s->batch), dim3(256), 0, st, a);
  return e;
}

}  // namespace kvs
