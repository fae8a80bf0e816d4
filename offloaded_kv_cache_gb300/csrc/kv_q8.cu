// kv_q8.cu -- the 8-bit paged cache: chunks of new tokens quantised as they
// are written, and pages read back into a cache of the model's own type.
//
// KVDrive (A Holistic Multi-Tier KV Cache Management System for Long-Context
// LLM Inference), section 2.3, and DirectKV (No Buffer, No Bottleneck),
// observation 4: what limits an offloaded cache is the bytes that cross
// the link.  e4m3 codes with one scale byte per vector are 129 bytes where
// 16-bit data takes 256.
//
// Both kernels move each byte once and compute a few operations per element,
// so memory bounds them; a decode step's append is bounded by latency.
#include <algorithm>

#include "kv_chunk.cuh"
#include "kv_launch.h"
#include "kv_q8.cuh"

namespace kvs {
namespace {

constexpr int kThreads = 256;
constexpr int kLanesPerVec = 16;  // 8 elements a lane: 16 bytes of 16-bit data, 8 bytes of codes

struct AppendArgs {
  const void *k_new, *v_new;
  uint8_t *k_codes, *v_codes, *k_scale, *v_scale;
  const int32_t *q_start, *bt, *ctx;
  int32_t *ctx_out;
  int *status;
  long long nphys;
  int B, Hkv, ps, maxP, total_q, max_q_len;
  int blocks;      // blocks per sequence
  int write_lens;  // this launch writes ctx_out
};

// A sequence's chunk: rows [q0, q0 + n), stored from position len on; n < 0
// when the sequence is skipped.
struct RowSpan {
  int q0, n, len;
};
__device__ __forceinline__ RowSpan append_span(const AppendArgs &a, int b) {
  const int q0 = a.q_start[b], q1 = a.q_start[b + 1], len = a.ctx[b];
  const long long cap = (long long)a.maxP * a.ps;
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.total_q && q1 - q0 <= a.max_q_len && len >= 0 &&
                  len + (long long)(q1 - q0) <= cap;
  return RowSpan{q0, ok ? q1 - q0 : -1, len};
}
// Whether every page the chunk touches is in range (the whole block asks).
__device__ __forceinline__ bool pages_ok(const AppendArgs &a, int b, const RowSpan &r) {
  bool bad = false;
  if (r.n > 0) {
    const int p0 = r.len / a.ps, p1 = (r.len + r.n - 1) / a.ps;
    for (int p = p0 + (int)threadIdx.x; p <= p1; p += blockDim.x) {
      const int ph = a.bt[(long long)b * a.maxP + p];
      bad |= ph < 0 || ph >= a.nphys;
    }
  }
  return !__syncthreads_or(bad);
}

// Block (b, j): vectors j, j + blocks, ... of the n_b * Hkv (token, head)
// pairs in steps of 16 vectors, K and V of each, so that two vectors per lane
// group are in flight.  Lengths: with one block per sequence, or with
// context_lens_out apart from context_lens, the sequence's first block writes
// them (every read of context_lens[b] in that block comes first); a chunk of
// several blocks updated in place takes a second launch (advance_kernel).
template <class T>
__global__ void __launch_bounds__(kThreads) q8_append_kernel(const AppendArgs a) {
  pdl_wait();
  const int b = blockIdx.x / a.blocks, j = blockIdx.x % a.blocks;
  const RowSpan r = append_span(a, b);
  if (j == 0) {
    const bool ok = r.n >= 0 && pages_ok(a, b, r);  // ends in a barrier when it asks
    if (threadIdx.x == 0) {
      if (!ok) flag_error(a.status, KV_ERR_BOUNDS);
      if (a.write_lens) a.ctx_out[b] = ok ? r.len + r.n : r.len;
    }
  }
  pdl_trigger();
  if (r.n <= 0) return;
  const int sub = threadIdx.x / kLanesPerVec, l = threadIdx.x % kLanesPerVec;
  constexpr int kVecs = kThreads / kLanesPerVec;
  const long long items = (long long)r.n * a.Hkv;
  const uint32_t half_mask = 0xFFFFu << (threadIdx.x & 16);
  const T *kn = static_cast<const T *>(a.k_new) + (long long)r.q0 * a.Hkv * kHeadDim;
  const T *vn = static_cast<const T *>(a.v_new) + (long long)r.q0 * a.Hkv * kHeadDim;
  for (long long it = (long long)j * kVecs + sub; it < items; it += (long long)a.blocks * kVecs) {
    const int i = (int)(it / a.Hkv), h = (int)(it % a.Hkv);
    const int pos = r.len + i;
    const int ph = a.bt[(long long)b * a.maxP + pos / a.ps];
    float x[2][8];
    load8(kn + it * kHeadDim + l * 8, x[0]);
    load8(vn + it * kHeadDim + l * 8, x[1]);
    if (ph < 0 || ph >= a.nphys) continue;  // recorded by the sequence's first block
    const long long vec = ((long long)ph * a.Hkv + h) * a.ps + pos % a.ps;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t top = 0;  // magnitudes order as their bits do, infinities and NaN above all
#pragma unroll
      for (int c = 0; c < 8; ++c) top = max(top, __float_as_uint(x[w][c]) & 0x7FFFFFFFu);
#pragma unroll
      for (int off = 8; off > 0; off >>= 1)
        top = max(top, __shfl_xor_sync(half_mask, top, off, kLanesPerVec));
      uint2 code = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
      int byte = kQ8NanScale;
      if (top < 0x7F800000u) {
        const int e = q8_exponent(top, q8_min_exp<T>());
        const float s = pow2f(-e);
        code.x = q8_codes4(x[w][0] * s, x[w][1] * s, x[w][2] * s, x[w][3] * s);
        code.y = q8_codes4(x[w][4] * s, x[w][5] * s, x[w][6] * s, x[w][7] * s);
        byte = e + 127;
      }
      *reinterpret_cast<uint2 *>((w ? a.v_codes : a.k_codes) + vec * kHeadDim + l * 8) = code;
      if (l == 0) (w ? a.v_scale : a.k_scale)[vec] = (uint8_t)byte;
    }
  }
}

// lengths of a chunk append in place, after every block has read them
__global__ void __launch_bounds__(kThreads) advance_kernel(const AppendArgs a) {
  pdl_wait();
  const int b = blockIdx.x;
  const RowSpan r = append_span(a, b);
  const bool ok = r.n >= 0 && pages_ok(a, b, r);
  __syncthreads();
  if (threadIdx.x == 0 && ok) a.ctx_out[b] = r.len + r.n;
}

struct ReadArgs {
  const uint8_t *codes[2], *scale[2];  // K, V
  void *out[2];
  const int32_t *bt, *ctx, *out_table;
  int *status;
  long long nphys, out_pages;
  int Hkv, ps, maxP;
  int tiles;  // 16-token tiles of a row: maxP * ps / 16
};

// Work item: (b, 16-token tile, kv head), 16 x 128 codes of K and of V.  A
// lane takes 8 codes and writes 8 elements, so that a half-warp reads and
// writes whole vectors; a block takes kUnits items, all loads issued before
// the first store.
constexpr int kUnits = 4;
template <class T>
__global__ void __launch_bounds__(kThreads) q8_read_kernel(const ReadArgs a, long long items) {
  pdl_wait();
  const int t = threadIdx.x / kLanesPerVec, l = threadIdx.x % kLanesPerVec;
  uint2 code[kUnits][2];
  uint32_t byte[kUnits][2];
  long long dst[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const long long it = (long long)blockIdx.x * kUnits + u;
    dst[u] = -1;
    if (it >= items) continue;
    const int h = (int)(it % a.Hkv);
    const long long bt_tile = it / a.Hkv;
    const int tile = (int)(bt_tile % a.tiles), b = (int)(bt_tile / a.tiles);
    const int len = a.ctx[b];
    const int pos = tile * kTileTokens + t, page = tile * kTileTokens / a.ps;
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
    const long long in = ((long long)src * a.Hkv + h) * a.ps + pos % a.ps;
    dst[u] = ((long long)to * a.Hkv + h) * a.ps + pos % a.ps;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      code[u][w] = *reinterpret_cast<const uint2 *>(a.codes[w] + in * kHeadDim + l * 8);
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
      store8(static_cast<T *>(a.out[w]) + dst[u] * kHeadDim + l * 8, x);
    }
  }
}

// Pages a chunk attention needs, brought into device memory in 16 bits:
// from the 8-bit cache, or from one in host memory.  Item and lanes as above.
struct StageArgs {
  const void *src[2];  // K, V: 16-bit data or codes
  const uint8_t *scale[2];
  void *out[2];
  const int32_t *q_start, *bt, *ctx;
  int32_t *table;  // [B][maxP] page in out, or null: the source's own page numbers
  int *status;
  long long nphys;
  int Hkv, ps, maxP, tiles, total_q, max_q_len, window;
};
template <class T, bool Q8>
__global__ void __launch_bounds__(kThreads) stage_kernel(const StageArgs a, long long items) {
  pdl_wait();
  const int t = threadIdx.x / kLanesPerVec, l = threadIdx.x % kLanesPerVec;
  uint4 data[kUnits][2];  // 16-bit data, or the codes in the first half
  uint32_t byte[kUnits][2];
  long long dst[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const long long it = (long long)blockIdx.x * kUnits + u;
    dst[u] = -1;
    if (it >= items) continue;
    const int h = (int)(it % a.Hkv);
    const long long bt_tile = it / a.Hkv;
    const int tile = (int)(bt_tile % a.tiles), b = (int)(bt_tile / a.tiles);
    const int tok0 = tile * kTileTokens, pos = tok0 + t, page = tok0 / a.ps;
    const int q0 = a.q_start[b], q1 = a.q_start[b + 1], len = a.ctx[b];
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
    const long long in = ((long long)src * a.Hkv + h) * a.ps + pos % a.ps;
    dst[u] = a.table ? (row * a.Hkv + h) * a.ps + pos % a.ps : in;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if constexpr (Q8) {
        const uint2 c = *reinterpret_cast<const uint2 *>(
            static_cast<const uint8_t *>(a.src[w]) + in * kHeadDim + l * 8);
        data[u][w] = make_uint4(c.x, c.y, 0, 0);
        byte[u][w] = a.scale[w][in];
      } else {
        data[u][w] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.src[w]) +
                                                      in * kHeadDim + l * 8);
      }
    }
  }
  pdl_trigger();
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    if (dst[u] < 0) continue;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      T *to = static_cast<T *>(a.out[w]) + dst[u] * kHeadDim + l * 8;
      if constexpr (Q8) {
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

cudaError_t launch_chunk_stage(int dtype, bool q8, const ChunkArgs &c, void *k_out, void *v_out,
                               int32_t *table, cudaStream_t st) {
  StageArgs a = {};
  a.src[0] = c.k;
  a.src[1] = c.v;
  a.scale[0] = c.k_scale;
  a.scale[1] = c.v_scale;
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
  a.maxP = c.maxP;
  a.tiles = (int)((long long)c.maxP * c.ps / kTileTokens);
  a.total_q = c.total_q;
  a.max_q_len = c.max_q_len;
  a.window = c.window;
  const long long items = (long long)c.B * a.tiles * a.Hkv;
  const long long blocks = (items + kUnits - 1) / kUnits;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(kThreads);
  if (dtype == KV_F16)
    return q8 ? launch_pdl(stage_kernel<__half, true>, grid, block, 0, st, a, items)
              : launch_pdl(stage_kernel<__half, false>, grid, block, 0, st, a, items);
  return q8 ? launch_pdl(stage_kernel<__nv_bfloat16, true>, grid, block, 0, st, a, items)
            : launch_pdl(stage_kernel<__nv_bfloat16, false>, grid, block, 0, st, a, items);
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
  a.maxP = maxP;
  a.total_q = total_q;
  a.max_q_len = max_q_len;
  // two steps of 16 vectors per block, up to a grid of 2^30 blocks
  const long long items = (long long)std::min(max_q_len, total_q) * Hkv;
  long long blocks = (items + 31) / 32;
  blocks = std::max(1LL, std::min(blocks, (1LL << 30) / B));
  a.blocks = (int)blocks;
  const bool in_place = ctx_out && ctx_out < ctx + B && ctx < ctx_out + B;
  const bool later = in_place && blocks > 1;
  a.write_lens = ctx_out && !later;
  const dim3 grid((unsigned)(blocks * B)), block(kThreads);
  cudaError_t e = dtype == KV_F32 ? launch_pdl(q8_append_kernel<float>, grid, block, 0, st, a)
                  : dtype == KV_F16
                      ? launch_pdl(q8_append_kernel<__half>, grid, block, 0, st, a)
                      : launch_pdl(q8_append_kernel<__nv_bfloat16>, grid, block, 0, st, a);
  if (e == cudaSuccess && later) e = launch_pdl(advance_kernel, dim3(B), block, 0, st, a);
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
  a.maxP = maxP;
  a.tiles = (int)((long long)maxP * ps / kTileTokens);
  const long long items = (long long)B * a.tiles * Hkv;
  const long long blocks = (items + kUnits - 1) / kUnits;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(kThreads);
  return dtype == KV_F32   ? launch_pdl(q8_read_kernel<float>, grid, block, 0, st, a, items)
         : dtype == KV_F16 ? launch_pdl(q8_read_kernel<__half>, grid, block, 0, st, a, items)
                           : launch_pdl(q8_read_kernel<__nv_bfloat16>, grid, block, 0, st, a, items);
}

}  // namespace kvs
