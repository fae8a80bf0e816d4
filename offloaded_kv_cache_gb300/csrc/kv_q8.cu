// kv_q8.cu -- the 8-bit paged cache: chunks of new tokens quantised as they
// are written, and pages read back into a cache of the model's own type.
//
// KVDrive (A Holistic Multi-Tier KV Cache Management System for Long-Context
// LLM Inference), section 2.3, and DirectKV (No Buffer, No Bottleneck),
// observation 4: what limits an offloaded cache is the bytes that cross
// the link.  e4m3 codes with one scale byte per vector are 129 bytes where
// 16-bit data takes 256.
//
// Both kernels move each byte once and compute a few operations per element, few
// enough to let memory bound them; a decode step's append is bounded by latency.
// Measured on one GB300, where a copy reaches 6.68 TB/s, replayed from graphs (as Python
// calls the short ones take what the host does, in brackets): append of 32 chunks of up
// to 513 tokens, 32 kv heads, f16: 30.3 us, 5.7 TB/s (computed in fp32, with divisions and
// each vector's maximum on its own: 35.0), fp32 data 47.6 us, 6.1 TB/s; of 4 x 2048 tokens,
// 8 kv heads: 6.4 us [21], fp32 12.4; of one token for 32 sequences: 2.1 us [16], fp32
// 2.3; read back of 4 x 32768 tokens, 8 kv heads, bf16: 105 us, 6.3 TB/s; of 4 x 16384
// into fp32: 103 us, 5.4 TB/s; of 2 x 544, 32 kv heads: 5.6 us [9.5], fp32 13.3.  The cache
// in pinned host memory: append of 4 x 2048 53 us, of 32 x 513 371 us, 156-160 GB/s of the
// link's 211 (the scales are single bytes); read back of 4 x 32768 1058 us, 211 GB/s.
#include <algorithm>

#include "kv_append.cuh"
#include "kv_chunk.cuh"
#include "kv_launch.h"
#include "kv_q4.cuh"
#include "kv_q8.cuh"

namespace kvs {
namespace {

constexpr int kThreads = 256;
#ifndef KVS_APPEND_BLOCKS
#define KVS_APPEND_BLOCKS 2432  // 16 per SM; 8: 32.1 us, 32: 31.1 us where this takes 30.3
#endif
constexpr int kLanesPerVec = 16;  // 8 elements a lane: 16 bytes of 16-bit data, 8 bytes of codes

struct AppendArgs {
  const void *k_new, *v_new;
  uint8_t *k_codes, *v_codes, *k_scale, *v_scale;
  const int32_t *q_start, *bt, *ctx;
  int32_t *ctx_out;
  int *status;
  long long nphys;
  int B, Hkv, ps, ps_log2, maxP, total_q, max_q_len;
  int blocks;      // blocks per sequence
  Divisor by_blocks, by_heads;
  int write_lens;  // this launch writes ctx_out
};

// Block (b, j) walks the n_b * Hkv (token, head) pairs of its sequence in steps
// of kSteps * 16, K and V of each pair, sixteen lanes a vector; the next step's
// loads are issued before this step's vectors are quantised, so that the
// round trips to the lengths and to the data are paid once per block and not
// once per step.  Lengths: with one block per sequence, or with context_lens_out
// apart from context_lens, the sequence's first block writes them (every read
// of context_lens[b] in that block comes first); a chunk of several blocks
// updated in place takes a second launch (advance_kernel).
constexpr int kVecs = kThreads / kLanesPerVec;
constexpr int kSteps = 2;
template <class T> struct AppendStep {
  uint4 w[kSteps][2][sizeof(T) / 2];
  int page[kSteps], pos[kSteps];
};
template <class T>
__global__ void __launch_bounds__(kThreads) q8_append_kernel(const AppendArgs a) {
  pdl_wait();
  const int b = a.by_blocks(blockIdx.x), j = (int)blockIdx.x - b * a.blocks;
  const RowSpan r = append_span(a, b);
  const int sub = threadIdx.x / kLanesPerVec, l = threadIdx.x % kLanesPerVec;
  const int items = r.n > 0 ? r.n * a.Hkv : 0;  // <= total_q * Hq, an int32
  const long long row0 = (long long)r.q0 * a.Hkv * kHeadDim + l * 8;
  const T *src[2] = {static_cast<const T *>(a.k_new) + row0,
                     static_cast<const T *>(a.v_new) + row0};
  auto load = [&](AppendStep<T> &s, long long step) {
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const long long it = step * (kVecs * kSteps) + u * kVecs + sub;
      s.page[u] = -1;
      if (it >= items) continue;
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int c = 0; c < (int)sizeof(T) / 2; ++c)
          s.w[u][w][c] = reinterpret_cast<const uint4 *>(src[w] + it * kHeadDim)[c];
      s.pos[u] = r.len + a.by_heads((int)it);
      s.page[u] = a.bt[(long long)b * a.maxP + (s.pos[u] >> a.ps_log2)];
    }
  };
  AppendStep<T> now;
  load(now, j);
  if (j == 0) {
    const bool ok = r.n >= 0 && pages_ok(a, b, r);  // ends in a barrier when it asks
    if (threadIdx.x == 0) {
      if (!ok) flag_error(a.status, KV_ERR_BOUNDS);
      if (a.write_lens) a.ctx_out[b] = ok ? r.len + r.n : r.len;
    }
  }
  pdl_trigger();
  const uint32_t half_mask = 0xFFFFu << (threadIdx.x & 16);
  for (long long step = j; step * (kVecs * kSteps) < items; step += a.blocks) {
    AppendStep<T> next;
    load(next, step + a.blocks);
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      // (a page out of range was recorded by the sequence's first block)
      if (now.page[u] < 0 || now.page[u] >= a.nphys) continue;
      const int it = (int)step * (kVecs * kSteps) + u * kVecs + sub;
      const int h = it - (now.pos[u] - r.len) * a.Hkv;
      // (rows of the cache fit int32)
      const long long vec = (now.page[u] * a.Hkv + h) * a.ps + (now.pos[u] & (a.ps - 1));
      uint32_t tops[2] = {q8_top(now.w[u][0]), q8_top(now.w[u][1])};
      if constexpr (sizeof(T) == 2) {  // K's and V's go through the lanes together
        uint32_t both = tops[0] | (tops[1] << 16);
#pragma unroll
        for (int off = 8; off > 0; off >>= 1)
          both = __vmaxu2(both, __shfl_xor_sync(half_mask, both, off, kLanesPerVec));
        tops[0] = both & 0xFFFFu;
        tops[1] = both >> 16;
      } else {
#pragma unroll
        for (int off = 8; off > 0; off >>= 1)
#pragma unroll
          for (int w = 0; w < 2; ++w)
            tops[w] = max(tops[w], __shfl_xor_sync(half_mask, tops[w], off, kLanesPerVec));
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t top = q8_top_f32(tops[w], T{});
        uint2 code = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        int byte = kQ8NanScale;
        if (top < 0x7F800000u) {
          const int e = q8_exponent(top, q8_min_exp<T>());
          code = q8_codes8(now.w[u][w], e, T{});
          byte = e + 127;
        }
        *reinterpret_cast<uint2 *>((w ? a.v_codes : a.k_codes) + vec * kHeadDim + l * 8) = code;
        if (l == 0) (w ? a.v_scale : a.k_scale)[vec] = (uint8_t)byte;
      }
    }
    now = next;
  }
}

struct ReadArgs {
  const uint8_t *codes[2], *scale[2];  // K, V
  void *out[2];
  const int32_t *bt, *ctx, *out_table;
  int *status;
  long long nphys, out_pages;
  int Hkv, ps, ps_log2, maxP;
  int items;   // of a sequence: (16-token tile, kv head) pairs
  int blocks;  // per sequence
  Divisor by_blocks, by_heads;
};

// Work item: (b, 16-token tile, kv head), 16 x 128 codes of K and of V.  A
// lane takes 8 codes and writes 8 elements, so that a half-warp reads and
// writes whole vectors; a block takes kUnits items, all loads issued before
// the first store.
constexpr int kUnits = 2;
template <class T>
__global__ void __launch_bounds__(kThreads) q8_read_kernel(const ReadArgs a) {
  pdl_wait();
  const int t = threadIdx.x / kLanesPerVec, l = threadIdx.x % kLanesPerVec;
  const int b = a.by_blocks(blockIdx.x), j = (int)blockIdx.x - b * a.blocks;
  const int len = a.ctx[b];
  uint2 code[kUnits][2];
  uint32_t byte[kUnits][2];
  int dst[kUnits];  // (rows of a cache fit int32)
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int it = j * kUnits + u;
    dst[u] = -1;
    if (it >= a.items) continue;
    const int tile = a.by_heads(it), h = it - tile * a.Hkv;
    const int pos = tile * kTileTokens + t, page = (tile * kTileTokens) >> a.ps_log2;
    if (len < 0 || (long long)len > (long long)a.maxP * a.ps) {
      if (threadIdx.x == 0 && tile == 0) flag_error(a.status, KV_ERR_BOUNDS);
      continue;
    }
    if (tile * kTileTokens >= len) continue;
    const long long row = (long long)b * a.maxP + page;
    const int src = a.bt[row], to = a.out_table[row];
    if (to < 0) continue;
    if (src < 0 || src >= a.nphys || to >= a.out_pages) {
      if (threadIdx.x == 0) flag_error(a.status, KV_ERR_BOUNDS);
      continue;
    }
    if (pos >= len) continue;
    const int in = (src * a.Hkv + h) * a.ps + (pos & (a.ps - 1));
    dst[u] = (to * a.Hkv + h) * a.ps + (pos & (a.ps - 1));
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      code[u][w] = *reinterpret_cast<const uint2 *>(a.codes[w] + (long long)in * kHeadDim + l * 8);
      byte[u][w] = a.scale[w][in];
    }
  }
  pdl_trigger();
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    if (dst[u] < 0) continue;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float lo[4], hi[4], x[8];
      q8_unpack4(code[u][w].x, lo);
      q8_unpack4(code[u][w].y, hi);
      const float s = q8_scale(byte[u][w]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[c] = lo[c] * s;
        x[4 + c] = hi[c] * s;
      }
      store8(static_cast<T *>(a.out[w]) + (long long)dst[u] * kHeadDim + l * 8, x);
    }
  }
}

// Pages a chunk attention needs, brought into device memory in T: from the 8-bit or
// the 4-bit cache, or from a 16-bit one in host memory.  Item and lanes as above.
struct StageArgs {
  const void *src[2];  // K, V: 16-bit data or codes
  const uint8_t *scale[2], *group[2];  // 8-bit: scales; 4-bit: powers and scales
  void *out[2];
  const int32_t *q_start, *bt, *ctx;
  int32_t *table;  // [B][maxP] page in out, or null: the source's own page numbers
  int *status;
  long long nphys;
  int Hkv, ps, ps_log2, maxP, items, blocks, total_q, max_q_len, window;
  Divisor by_blocks, by_heads;
};
template <class T, CacheForm kForm>
__global__ void __launch_bounds__(kThreads) stage_kernel(const StageArgs a) {
  pdl_wait();
  const int t = threadIdx.x / kLanesPerVec, l = threadIdx.x % kLanesPerVec;
  const int b = a.by_blocks(blockIdx.x), j = (int)blockIdx.x - b * a.blocks;
  const int q0 = a.q_start[b], q1 = a.q_start[b + 1], len = a.ctx[b];
  uint4 data[kUnits][2];  // 16-bit data, or the codes and what they need
  uint32_t byte[kUnits][2];
  int dst[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int it = j * kUnits + u;
    dst[u] = -1;
    if (it >= a.items) continue;
    const int tile = a.by_heads(it), h = it - tile * a.Hkv;
    const int tok0 = tile * kTileTokens, pos = tok0 + t, page = tok0 >> a.ps_log2;
    // sequences the attention skips (and records), and tokens no row sees
    if (q0 < 0 || q1 <= q0 || q1 > a.total_q || q1 - q0 > a.max_q_len || len < 0 ||
        (long long)len > (long long)a.maxP * a.ps || tok0 >= len)
      continue;
    if (a.window > 0 &&
        (long long)(tok0 / kChunkTile + 1) * kChunkTile <= (long long)len - (q1 - q0) - a.window + 1)
      continue;
    const long long row = (long long)b * a.maxP + page;
    const int src = a.bt[row];
    const bool ok = src >= 0 && src < a.nphys;
    if (a.table && h == 0 && threadIdx.x == 0 && tok0 % a.ps == 0)
      a.table[row] = ok ? (int32_t)row : -1;
    if (!ok || pos >= len) continue;
    const int in = (src * a.Hkv + h) * a.ps + (pos & (a.ps - 1));
    dst[u] = a.table ? ((int)row * a.Hkv + h) * a.ps + (pos & (a.ps - 1)) : in;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if constexpr (kForm == kQ4Form) {
        data[u][w].x = *reinterpret_cast<const uint32_t *>(
            static_cast<const uint8_t *>(a.src[w]) + (long long)in * kQ4Bytes + l * 4);
        data[u][w].y = a.group[w][(long long)in * kQ4Scales + l / 2];
        byte[u][w] = a.scale[w][in];
      } else if constexpr (kForm == kQ8Form) {
        const uint2 c = *reinterpret_cast<const uint2 *>(
            static_cast<const uint8_t *>(a.src[w]) + (long long)in * kHeadDim + l * 8);
        data[u][w] = make_uint4(c.x, c.y, 0, 0);
        byte[u][w] = a.scale[w][in];
      } else {
        data[u][w] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.src[w]) +
                                                      (long long)in * kHeadDim + l * 8);
      }
    }
  }
  pdl_trigger();
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    if (dst[u] < 0) continue;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      T *to = static_cast<T *>(a.out[w]) + (long long)dst[u] * kHeadDim + l * 8;
      if constexpr (kForm == kQ4Form) {
        q4_store8(to, data[u][w].x, e4m3_pair(data[u][w].y).x * q4_power(byte[u][w]), Q4Bits<T>());
      } else if constexpr (kForm == kQ8Form) {
        float lo[4], hi[4], x[8];
        q8_unpack4(data[u][w].x, lo);
        q8_unpack4(data[u][w].y, hi);
        const float s = q8_scale(byte[u][w]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[c] = lo[c] * s;
          x[4 + c] = hi[c] * s;
        }
        store8(to, x);
      } else {
        *reinterpret_cast<uint4 *>(to) = data[u][w];
      }
    }
  }
}

}  // namespace

namespace {
// (16-token tile, kv head) items of a sequence, and the blocks they take
bool item_grid(int B, int maxP, int ps, int Hkv, int *items, int *blocks) {
  const long long n = (long long)maxP * ps / kTileTokens * Hkv, k = (n + kUnits - 1) / kUnits;
  if (n > 0x7FFFFFFFLL - kUnits || k * B > 0x7FFFFFFFLL) return false;
  *items = (int)n;
  *blocks = (int)k;
  return true;
}
}  // namespace

bool q8_grid_fits(int B, int maxP, int ps, int Hkv) {
  int items, blocks;
  return item_grid(B, maxP, ps, Hkv, &items, &blocks);
}

cudaError_t launch_chunk_stage(int dtype, CacheForm form, const ChunkArgs &c, void *k_out,
                               void *v_out, int32_t *table, cudaStream_t st) {
  StageArgs a = {};
  a.src[0] = c.k;
  a.src[1] = c.v;
  a.scale[0] = c.k_scale;
  a.scale[1] = c.v_scale;
  a.group[0] = c.k_group;
  a.group[1] = c.v_group;
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.q_start = c.q_start;
  a.bt = c.bt;
  a.ctx = c.ctx;
  a.table = table;
  a.status = c.status;
  a.nphys = c.nphys;
  a.Hkv = c.Hkv;
  a.ps = c.ps;
  a.ps_log2 = __builtin_ctz(c.ps);
  a.maxP = c.maxP;
  a.total_q = c.total_q;
  a.max_q_len = c.max_q_len;
  a.window = c.window;
  if (!item_grid(c.B, c.maxP, c.ps, c.Hkv, &a.items, &a.blocks))
    return cudaErrorInvalidConfiguration;
  a.by_blocks = Divisor::of(a.blocks);
  a.by_heads = Divisor::of(c.Hkv);
  const dim3 grid((unsigned)(a.blocks * c.B)), block(kThreads);
  if (dtype == KV_F32) return launch_pdl(stage_kernel<float, kQ4Form>, grid, block, 0, st, a);
  if (dtype == KV_F16)
    return form == kQ4Form   ? launch_pdl(stage_kernel<__half, kQ4Form>, grid, block, 0, st, a)
           : form == kQ8Form ? launch_pdl(stage_kernel<__half, kQ8Form>, grid, block, 0, st, a)
                             : launch_pdl(stage_kernel<__half, kOwnForm>, grid, block, 0, st, a);
  return form == kQ4Form   ? launch_pdl(stage_kernel<__nv_bfloat16, kQ4Form>, grid, block, 0, st, a)
         : form == kQ8Form ? launch_pdl(stage_kernel<__nv_bfloat16, kQ8Form>, grid, block, 0, st, a)
                           : launch_pdl(stage_kernel<__nv_bfloat16, kOwnForm>, grid, block, 0, st, a);
}

cudaError_t launch_q8_append(int dtype, const void *k_new, const void *v_new,
                             const kv_q8_cache &c, const int32_t *q_start, const int32_t *bt,
                             const int32_t *ctx, int32_t *ctx_out, int B, int Hkv, int ps,
                             int maxP, long long nphys, int total_q, int max_q_len, int *status,
                             cudaStream_t st) {
  AppendArgs a = {};
  a.k_new = k_new;
  a.v_new = v_new;
  a.k_codes = c.k_codes;
  a.v_codes = c.v_codes;
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.q_start = q_start;
  a.bt = bt;
  a.ctx = ctx;
  a.ctx_out = ctx_out;
  a.status = status;
  a.nphys = nphys;
  a.B = B;
  a.Hkv = Hkv;
  a.ps = ps;
  a.ps_log2 = __builtin_ctz(ps);
  a.maxP = maxP;
  a.total_q = total_q;
  a.max_q_len = max_q_len;
  const long long items = (long long)std::min(max_q_len, total_q) * Hkv;
  // as many blocks as there are steps, up to what keeps every SM busy
  const long long steps = (items + kVecs * kSteps - 1) / (kVecs * kSteps);
  a.blocks = (int)std::max(1LL, std::min(steps, (KVS_APPEND_BLOCKS + B - 1LL) / B));
  a.by_blocks = Divisor::of(a.blocks);
  a.by_heads = Divisor::of(Hkv);
  const long long blocks = a.blocks;
  const bool later = ctx_out == ctx && blocks > 1;
  a.write_lens = ctx_out && !later;
  const dim3 grid((unsigned)(blocks * B)), block(kThreads);
  cudaError_t e = dtype == KV_F32 ? launch_pdl(q8_append_kernel<float>, grid, block, 0, st, a)
                  : dtype == KV_F16
                      ? launch_pdl(q8_append_kernel<__half>, grid, block, 0, st, a)
                      : launch_pdl(q8_append_kernel<__nv_bfloat16>, grid, block, 0, st, a);
  if (e == cudaSuccess && later) e = launch_pdl(advance_kernel<AppendArgs>, dim3(B), block, 0, st, a);
  return e;
}

cudaError_t launch_q8_read(int dtype, const kv_q8_cache &c, const int32_t *bt, const int32_t *ctx,
                           const int32_t *out_table, long long out_pages, void *k_out,
                           void *v_out, int B, int Hkv, int ps, int maxP, long long nphys,
                           int *status, cudaStream_t st) {
  ReadArgs a = {};
  a.codes[0] = c.k_codes;
  a.codes[1] = c.v_codes;
  a.scale[0] = c.k_scale;
  a.scale[1] = c.v_scale;
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
  if (!item_grid(B, maxP, ps, Hkv, &a.items, &a.blocks)) return cudaErrorInvalidConfiguration;
  a.by_blocks = Divisor::of(a.blocks);
  a.by_heads = Divisor::of(Hkv);
  const dim3 grid((unsigned)(a.blocks * B)), block(kThreads);
  return dtype == KV_F32   ? launch_pdl(q8_read_kernel<float>, grid, block, 0, st, a)
         : dtype == KV_F16 ? launch_pdl(q8_read_kernel<__half>, grid, block, 0, st, a)
                           : launch_pdl(q8_read_kernel<__nv_bfloat16>, grid, block, 0, st, a);
}

}  // namespace kvs
