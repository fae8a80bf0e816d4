// kv_q4.cu -- the 4-bit paged cache: chunks of new tokens quantised as they are written,
// and pages read back into a cache of the model's own type.  (The same bytes expanded for
// an attention that passes through the workspace: kv_q8.cu's staging.)
//
// 73 bytes a vector where 16-bit data takes 256: memory bounds the read back (4 x <= 32768
// tokens, 8 kv heads, bf16: 92 us, 568 MB, 6.2 TB/s), the append nearly: its issue slots are
// busy for some 70% of the time (32 x <= 513 tokens, 32 kv heads: f16 26 us, 148 MB, 5.6 TB/s;
// fp32 47 us, 5.6 TB/s).  A decode step's append (2.2 us) is the launch and two round trips.
#include <algorithm>
#include <type_traits>

#include "kv_append.cuh"
#include "kv_launch.h"
#include "kv_q4.cuh"

namespace kvs {
namespace {

constexpr int kThreads = 256;
constexpr int kLanesPerVec = 16;  // of the read back: 8 channels a lane, two lanes a scale
#ifndef KVS_APPEND4_BLOCKS
#define KVS_APPEND4_BLOCKS 2432  // 16 per SM
#endif

struct AppendArgs {
  const void *src[2];  // K, V
  uint8_t *codes[2], *scale[2], *power[2];
  const int32_t *q_start, *bt, *ctx;
  int32_t *ctx_out;
  int *status;
  long long nphys;
  int Hkv, ps, ps_log2, maxP, total_q, max_q_len;
  int blocks;  // per sequence
  Divisor by_blocks, by_heads;
  int write_lens;
};

// Block (b, j) walks the n_b * Hkv (token, head) pairs of its sequence, K and V of each pair;
// the next step's loads are issued before this step's vectors are quantised.  16-bit data: a
// lane has the 16 channels of a scale, eight lanes a vector, so that what is computed per scale
// and per vector is computed half as often (sixteen lanes a vector: 32 x 513 tokens, 32 kv
// heads, 36 us).  fp32: 8 channels, sixteen lanes, whose loads lie closer together.
template <class T> struct AppendStep {
  static constexpr int kChannels = sizeof(T) == 2 ? 16 : 8;  // of a lane
  static constexpr int kLanes = kHeadDim / kChannels, kVecs = kThreads / kLanes;
  static constexpr int kLoads = kChannels * (int)sizeof(T) / 16;
  uint4 w[2][kLoads];
  int page, pos;
};
// The bits of the largest magnitude of sixteen 16-bit elements; of a NaN's where there is one.
// (As numbers: the absolute values cost nothing.)
template <class T> __device__ __forceinline__ uint32_t q4_top16(const uint4 (&w)[2], T) {
  using Two = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
  const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
  Two m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m[i] = __hmax2_nan(__habs2(reinterpret_cast<const Two &>(u[i])), __habs2(reinterpret_cast<const Two &>(u[i + 4])));
  const Two top = __hmax2_nan(__hmax2_nan(m[0], m[1]), __hmax2_nan(m[2], m[3]));
  const uint32_t t = reinterpret_cast<const uint32_t &>(top);
  return max(t & 0xFFFFu, t >> 16);
}
__device__ __forceinline__ uint32_t q4_top32(const uint4 (&w)[2]) {  // of eight fp32 elements
  const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
  float m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = fabsf(__uint_as_float(u[i]));
#pragma unroll
  for (int n = 4; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m[i]) : "f"(m[i + n]));
  return __float_as_uint(m[0]);
}
template <class T>
__global__ void __launch_bounds__(kThreads) q4_append_kernel(const AppendArgs a) {
  using Step = AppendStep<T>;
  constexpr int kLanes = Step::kLanes, kVecs = Step::kVecs, kChannels = Step::kChannels;
  pdl_wait();
  const int b = a.by_blocks(blockIdx.x), j = (int)blockIdx.x - b * a.blocks;
  const RowSpan r = append_span(a, b);
  const int sub = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
  const int items = r.n > 0 ? r.n * a.Hkv : 0;  // <= total_q * Hq, an int32
  const long long row0 = (long long)r.q0 * a.Hkv * kHeadDim + l * kChannels;
  const T *src[2] = {static_cast<const T *>(a.src[0]) + row0, static_cast<const T *>(a.src[1]) + row0};
  auto load = [&](Step &s, long long step) {
    const long long it = step * kVecs + sub;
    s.page = -1;
    s.pos = 0;
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int c = 0; c < Step::kLoads; ++c) s.w[w][c] = make_uint4(0, 0, 0, 0);
    if (it >= items) return;
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int c = 0; c < Step::kLoads; ++c)
        s.w[w][c] = reinterpret_cast<const uint4 *>(src[w] + it * kHeadDim)[c];
    s.pos = r.len + a.by_heads((int)it);
    s.page = a.bt[(long long)b * a.maxP + (s.pos >> a.ps_log2)];
  };
  Step now;
  load(now, j);
  if (j == 0) {
    const bool ok = r.n >= 0 && pages_ok(a, b, r);  // ends in a barrier when it asks
    if (threadIdx.x == 0) {
      if (!ok) flag_error(a.status, KV_ERR_BOUNDS);
      if (a.write_lens) a.ctx_out[b] = ok ? r.len + r.n : r.len;
    }
  }
  pdl_trigger();
  // (all lanes of a warp take part, those without a vector too)
  auto quantise = [&](const Step &s, long long step) {
    // the largest magnitude of the 16 channels of a scale, of the vector
    uint32_t group[2], top[2];
    if constexpr (sizeof(T) == 2) {  // K's and V's go through the lanes together
#pragma unroll
      for (int w = 0; w < 2; ++w)
        group[w] = q4_top16(s.w[w], T{});
      uint32_t both = group[0] | (group[1] << 16);
#pragma unroll
      for (int off = 1; off < kLanes; off <<= 1)
        both = __vmaxu2(both, __shfl_xor_sync(0xFFFFFFFFu, both, off));
      top[0] = both & 0xFFFFu;
      top[1] = both >> 16;
    } else {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        top[w] = q4_top32(s.w[w]);
        top[w] = group[w] = max(top[w], __shfl_xor_sync(0xFFFFFFFFu, top[w], 1));
#pragma unroll
        for (int off = 2; off < kLanes; off <<= 1)
          top[w] = max(top[w], __shfl_xor_sync(0xFFFFFFFFu, top[w], off));
      }
    }
    const int it = (int)step * kVecs + sub;
    const int h = it - (s.pos - r.len) * a.Hkv;
    // (rows of the cache fit int32)
    const int vec = (s.page * a.Hkv + h) * a.ps + (s.pos & (a.ps - 1));
    // (a page out of range was recorded by the sequence's first block)
    const bool there = s.page >= 0 && s.page < a.nphys;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint32_t most = q8_top_f32(top[w], T{});
      const int e = q4_exponent(most, q8_min_exp<T>());
      const float y = __uint_as_float(q8_top_f32(group[w], T{})) * pow2f(-e);
      float f;
      const uint32_t scale = q4_scale_code(y, f);
      uint32_t code[kChannels / 8];
#pragma unroll
      for (int c = 0; c < kChannels / 8; ++c) {
        float x[8];
        load8(reinterpret_cast<const T *>(s.w[w]) + 8 * c, x);
        code[c] = q4_codes8(x, y, f, e, T{});
      }
      if (!there) continue;
      const bool nan = most >= 0x7F800000u;
      uint8_t *to = a.codes[w] + (long long)vec * kQ4Bytes;
      if constexpr (kChannels == 16) {
        reinterpret_cast<uint2 *>(to)[l] =
            nan ? make_uint2(0x88888888u, 0x88888888u) : make_uint2(code[0], code[1]);
        a.scale[w][(long long)vec * kQ4Scales + l] = (uint8_t)(nan ? 0 : scale);
      } else {
        reinterpret_cast<uint32_t *>(to)[l] = nan ? 0x88888888u : code[0];
        if (!(l & 1)) a.scale[w][(long long)vec * kQ4Scales + l / 2] = (uint8_t)(nan ? 0 : scale);
      }
      if (l == 0) a.power[w][vec] = (uint8_t)(nan ? kQ4NanPower : e + 127);
    }
  };
  for (long long step = j; step * kVecs < items;) {
    Step next;
    load(next, step + a.blocks);
    quantise(now, step);
    step += a.blocks;
    if (step * kVecs >= items) break;
    load(now, step + a.blocks);
    quantise(next, step);
    step += a.blocks;
  }
}

struct ReadArgs {
  const uint8_t *codes[2], *scale[2], *power[2];
  void *out[2];
  const int32_t *bt, *ctx, *out_table;
  int *status;
  long long nphys, out_pages;
  int Hkv, ps, ps_log2, maxP;
  int blocks;  // per sequence
  Divisor by_blocks, by_heads;
};

// Work item: (b, 16-token tile, kv head), a half-warp per token and lanes as above.  Block (b,
// j) walks its sequence's items in steps of kUnits, the next step's codes in flight while this
// one's are stored, and the pages of the step after that looked up.  (A block for each step
// paid three dependent round trips by itself: 4 x 32768 tokens, 8 kv heads, bf16 102 us.)
#ifndef KVS_READ4_BLOCKS
#define KVS_READ4_BLOCKS 1216  // 8 per SM
#endif
constexpr int kUnits = 2;
struct ReadPages {
  int src[kUnits], to[kUnits];  // src < 0: nothing to do
};
struct ReadStep {
  uint32_t code[kUnits][2], scale[kUnits][2], byte[kUnits][2];
  int dst[kUnits];  // (rows of a cache fit int32)
};
template <class T>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(const ReadArgs a) {
  pdl_wait();
  const int t = threadIdx.x / kLanesPerVec, l = threadIdx.x % kLanesPerVec;
  const int b = a.by_blocks(blockIdx.x), j = (int)blockIdx.x - b * a.blocks;
  const int len = a.ctx[b];
  if (len < 0 || (long long)len > (long long)a.maxP * a.ps) {
    if (threadIdx.x == 0) flag_error(a.status, KV_ERR_BOUNDS);
    return;
  }
  // (tiles and heads of the block table's width count in int32)
  const int items = (len + kTileTokens - 1) / kTileTokens * a.Hkv, stride = a.blocks * kUnits;
  auto look_up = [&](ReadPages &p, long long it0) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      p.src[u] = -1;
      if (it0 + u >= items) continue;
      const long long row = (long long)b * a.maxP + ((a.by_heads((int)it0 + u) * kTileTokens) >> a.ps_log2);
      p.src[u] = a.bt[row];
      p.to[u] = a.out_table[row];
    }
  };
  auto load = [&](ReadStep &s, const ReadPages &p, long long it0) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      s.dst[u] = -1;
      if (it0 + u >= items || p.to[u] < 0) continue;
      if (p.src[u] < 0 || p.src[u] >= a.nphys || p.to[u] >= a.out_pages) {
        if (threadIdx.x == 0) flag_error(a.status, KV_ERR_BOUNDS);
        continue;
      }
      const int tile = a.by_heads((int)it0 + u), h = (int)it0 + u - tile * a.Hkv;
      const int pos = tile * kTileTokens + t;
      if (pos >= len) continue;
      const int in = (p.src[u] * a.Hkv + h) * a.ps + (pos & (a.ps - 1));
      s.dst[u] = (p.to[u] * a.Hkv + h) * a.ps + (pos & (a.ps - 1));
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint8_t *code = a.codes[w] + (long long)in * kQ4Bytes;
        const uint8_t *scale = a.scale[w] + (long long)in * kQ4Scales;
        if constexpr (sizeof(T) == 2) {
          s.code[u][w] = *reinterpret_cast<const uint32_t *>(code + 4 * l);
          s.scale[u][w] = scale[l / 2];
        } else {
          s.code[u][w] = *reinterpret_cast<const uint16_t *>(code + 2 * l) |
                         *reinterpret_cast<const uint16_t *>(code + 32 + 2 * l) << 16;
          s.scale[u][w] = scale[l / 4] | scale[4 + l / 4] << 8;
        }
        s.byte[u][w] = a.power[w][in];
      }
    }
  };
  const Q4Bits<T> bits;
  auto store = [&](const ReadStep &s) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (s.dst[u] < 0) continue;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        T *to = static_cast<T *>(a.out[w]) + (long long)s.dst[u] * kHeadDim;
        const float2 f = e4m3_pair(s.scale[u][w]);
        const float p = q4_power(s.byte[u][w]);
        if constexpr (sizeof(T) == 2) {
          q4_store8(to + l * 8, s.code[u][w], f.x * p, bits);
        } else {  // four channels of each half: a half-warp's stores have no gaps
          *reinterpret_cast<float4 *>(to + 4 * l) = q4_values4(s.code[u][w], f.x * p);
          *reinterpret_cast<float4 *>(to + 64 + 4 * l) = q4_values4(s.code[u][w] >> 16, f.y * p);
        }
      }
    }
  };
  ReadPages pages;
  ReadStep now, next;
  long long it = (long long)j * kUnits;
  look_up(pages, it);
  load(now, pages, it);
  look_up(pages, it + stride);
  pdl_trigger();
  while (it < items) {
    load(next, pages, it + stride);
    look_up(pages, it + 2 * stride);
    store(now);
    it += stride;
    if (it >= items) break;
    load(now, pages, it + stride);
    look_up(pages, it + 2 * stride);
    store(next);
    it += stride;
  }
}

}  // namespace

cudaError_t launch_q4_append(int dtype, const void *k_new, const void *v_new,
                             const kv_q4_cache &c, const int32_t *q_start, const int32_t *bt,
                             const int32_t *ctx, int32_t *ctx_out, int B, int Hkv, int ps,
                             int maxP, long long nphys, int total_q, int max_q_len, int *status,
                             cudaStream_t st) {
  AppendArgs a = {};
  a.src[0] = k_new;
  a.src[1] = v_new;
  a.codes[0] = c.k_codes;
  a.codes[1] = c.v_codes;
  a.scale[0] = c.k_scale;
  a.scale[1] = c.v_scale;
  a.power[0] = c.k_power;
  a.power[1] = c.v_power;
  a.q_start = q_start;
  a.bt = bt;
  a.ctx = ctx;
  a.ctx_out = ctx_out;
  a.status = status;
  a.nphys = nphys;
  a.Hkv = Hkv;
  a.ps = ps;
  a.ps_log2 = __builtin_ctz(ps);
  a.maxP = maxP;
  a.total_q = total_q;
  a.max_q_len = max_q_len;
  const long long items = (long long)std::min(max_q_len, total_q) * Hkv;
  const int vecs = dtype == KV_F32 ? AppendStep<float>::kVecs : AppendStep<__half>::kVecs;
  const long long steps = (items + vecs - 1) / vecs;
  a.blocks = (int)std::max(1LL, std::min(steps, (KVS_APPEND4_BLOCKS + B - 1LL) / B));
  a.by_blocks = Divisor::of(a.blocks);
  a.by_heads = Divisor::of(Hkv);
  const bool later = ctx_out == ctx && a.blocks > 1;
  a.write_lens = ctx_out && !later;
  const dim3 grid((unsigned)((long long)a.blocks * B)), block(kThreads);
  cudaError_t e = dtype == KV_F32 ? launch_pdl(q4_append_kernel<float>, grid, block, 0, st, a)
                  : dtype == KV_F16
                      ? launch_pdl(q4_append_kernel<__half>, grid, block, 0, st, a)
                      : launch_pdl(q4_append_kernel<__nv_bfloat16>, grid, block, 0, st, a);
  if (e == cudaSuccess && later) e = launch_pdl(advance_kernel<AppendArgs>, dim3(B), block, 0, st, a);
  return e;
}

cudaError_t launch_q4_read(int dtype, const kv_q4_cache &c, const int32_t *bt, const int32_t *ctx,
                           const int32_t *out_table, long long out_pages, void *k_out,
                           void *v_out, int B, int Hkv, int ps, int maxP, long long nphys,
                           int *status, cudaStream_t st) {
  ReadArgs a = {};
  a.codes[0] = c.k_codes;
  a.codes[1] = c.v_codes;
  a.scale[0] = c.k_scale;
  a.scale[1] = c.v_scale;
  a.power[0] = c.k_power;
  a.power[1] = c.v_power;
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.bt = bt;
  a.ctx = ctx;
  a.out_table = out_table;
  a.status = status;
  a.nphys = nphys;
  a.out_pages = out_pages;
  a.Hkv = Hkv;
  a.ps = ps;
  a.ps_log2 = __builtin_ctz(ps);
  a.maxP = maxP;
  // (the entry point has checked, by q8_grid_fits, that the items count in int32)
  const long long steps = ((long long)maxP * ps / kTileTokens * Hkv + kUnits - 1) / kUnits;
  a.blocks = (int)std::max(1LL, std::min(steps, (KVS_READ4_BLOCKS + B - 1LL) / B));
  a.by_blocks = Divisor::of(a.blocks);
  a.by_heads = Divisor::of(Hkv);
  const dim3 grid((unsigned)((long long)a.blocks * B)), block(kThreads);
  return dtype == KV_F32   ? launch_pdl(q4_read_kernel<float>, grid, block, 0, st, a)
         : dtype == KV_F16 ? launch_pdl(q4_read_kernel<__half>, grid, block, 0, st, a)
                           : launch_pdl(q4_read_kernel<__nv_bfloat16>, grid, block, 0, st, a);
}

}  // namespace kvs
