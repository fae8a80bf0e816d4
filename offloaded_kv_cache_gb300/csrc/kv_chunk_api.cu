// kv_chunk_api.cu -- the extern "C" boundary of the chunk operators: argument
// checks, launch plans and launches.  Contracts are in include/kvsparse.h.
#include <algorithm>
#include <climits>
#include <cmath>

#include "kv_chunk.cuh"
#include "kv_host.h"
#include "kv_launch.h"

namespace {

using namespace kvs;

int check_chunk(const kv_shape *s, const kv_chunk *c) {
  if (!c || !al4(c->q_start) || c->total_q < 1 || c->max_q_len < 1 || c->window < 0 ||
      c->reserved != 0)
    return KV_ERR_INVALID_ARG;
  // packed rows (token, head of the group) and output rows fit in int32
  if ((long long)c->total_q * s->num_q_heads > INT_MAX) return KV_ERR_UNSUPPORTED;
  return KV_OK;
}

// The four arrays of an 8-bit cache, as the device sees them.
int resolve_q8(const kv_shape *s, const kv_q8_cache *c, kv_q8_cache *dev) {
  if (!c) return KV_ERR_INVALID_ARG;
  const uint8_t *const in[4] = {c->k_codes, c->v_codes, c->k_scale, c->v_scale};
  const void *out[4];
  for (int i = 0; i < 4; ++i) {
    const int rc = resolve_kv(s, in[i], &out[i]);
    if (rc != KV_OK) return rc;
  }
  dev->k_codes = static_cast<uint8_t *>(const_cast<void *>(out[0]));
  dev->v_codes = static_cast<uint8_t *>(const_cast<void *>(out[1]));
  dev->k_scale = static_cast<uint8_t *>(const_cast<void *>(out[2]));
  dev->v_scale = static_cast<uint8_t *>(const_cast<void *>(out[3]));
  return KV_OK;
}

// The six arrays of a 4-bit cache, likewise.
int resolve_q4(const kv_shape *s, const kv_q4_cache *c, kv_q4_cache *dev) {
  if (!c) return KV_ERR_INVALID_ARG;
  uint8_t *const in[6] = {c->k_codes, c->v_codes, c->k_scale, c->v_scale, c->k_power, c->v_power};
  uint8_t **const to[6] = {&dev->k_codes, &dev->v_codes, &dev->k_scale,
                           &dev->v_scale, &dev->k_power, &dev->v_power};
  for (int i = 0; i < 6; ++i) {
    const void *at;
    const int rc = resolve_kv(s, in[i], &at);
    if (rc != KV_OK) return rc;
    *to[i] = static_cast<uint8_t *>(const_cast<void *>(at));
  }
  return KV_OK;
}

// Up to this many packed rows the 16-bit kernels' converting form reads the
// 8-bit cache itself, in units of 128 rows; above, the cache is expanded into the
// workspace first and read in units of 256.  (4 x 32k tokens, 8 kv heads, us,
// direct / expanded, bf16: 128 rows 78 / 175, 256 rows 111 / 186, 512 rows 183 /
// 215, 640 rows 217 / 238; f16: 640 rows 189 / 239.)
#ifndef KVS_Q8_DIRECT_ROWS
#define KVS_Q8_DIRECT_ROWS 768
#endif
// The 4-bit cache likewise.  (us, direct / expanded, 8 kv heads: 4 x 32k tokens in pages of 16,
// bf16, 128 rows 81 / 168, 512 rows 201 / 209, 1024 rows 362 / 289; in pages of 64, 512 rows 170 /
// 205, 1024 rows 309 / 288; 16 x 2k, f16, 512 rows 56 / 66, 1024 rows 89 / 85.)
#ifndef KVS_Q4_DIRECT_ROWS
#define KVS_Q4_DIRECT_ROWS 640
#endif
// What a row may see, as far as the host knows.
long long seen_tokens(const kv_shape *s, int window) {
  const long long tokens = (long long)s->max_pages_per_seq * s->page_size;
  return window > 0 ? std::min<long long>(tokens, window) : tokens;
}
// 16-bit K/V on the tensor cores: while a row sees few tokens the loads of Q, the
// diagonal and the way out are most of a unit, and two CTAs with a unit of 128
// rows each cover them for one another (kSolo); over long contexts units of 256
// rows read K and V half as often (kWide), and few rows keep more of the stream in
// flight with an SM's whole memory (kPair).  us, two CTAs / one, bf16: 32 prompts of
// 512, 32/32 heads 82 / 95, of 800 142 / 155, of 1000 194 / 195, of 1400 336 / 290;
// 4 of 800, 64/8 heads 54 / 52; 20 new tokens over 32 x 1000, 32/32 heads 61 / 68;
// 32/8 heads, over 32 x 4000 66 / 73, over 32 x 8000 110 / 120, over 1 x 8000 31 / 25.
#ifndef KVS_SOLO_TOKENS
#define KVS_SOLO_TOKENS 896
#endif
#ifndef KVS_SOLO_FEW
#define KVS_SOLO_FEW 4096
#endif
// Up to this many packed rows the kernel for few rows is taken (kv_chunk_few.cu,
// units of 8 that each read K and V).  Its reads cost more the longer what a row
// sees may be, which the host knows by the block table's width and the window.
// For fp32 q over the 8-bit cache the other kernel computes on the CUDA cores:
// only many rows that see little are left to that one.  us, few / the other
// kernel, 8 kv heads, bf16 q:
//   8-bit, 4 x 32k tokens: 8 rows 43 / 69, 16 rows 66 / 69, 24 rows 89 / 70;
//     16 x 2k: 16 rows 22 / 27, 24 rows 26 / 27; 17 x 456, 32 kv heads: 24 rows 31 / 38
//   16-bit, 4 x 32k: 8 rows 66 / 68, 16 rows 100 / 68; 16 x 2k: 16 rows 24.5 / 26.7,
//     24 rows 29.7 / 26.9; 17 x 456, 32 kv heads: 8 rows 24 / 34, 16 rows 30 / 35
//   fp32 q, 8-bit, 4 x 32k: 8 rows 70 / 410, 16 rows 106 / 655; 4 x 1.9k: 256 rows
//     74 / 132; 8448 rows over 528, 2 kv heads: 289 / 112; window 90, 880 rows: 104 / 53
//   4-bit (kv_chunk_q4.cu), 4 x 32k: 16 rows 47 / 74, 24 rows 54 / 74, 32 rows 80 / 75; 16 x 2k,
//     f16: 24 rows 26 / 27, 32 rows 28 / 27; 17 x 456, 32 kv heads: 16 rows 25 / 35, 32 rows 36 /
//     36.  fp32 q (the other kernel reads a copy in fp32): 4 x 32k: 8 rows 40 / 356, 64 rows 164 /
//     798; 4 x 8k: 2048 rows 1209 / 3307; 16 x 500: 64 rows 23 / 75, 1024 rows 266 / 342
int few_rows_limit(const kv_shape *s, int window, CacheForm form) {
  const long long seen = seen_tokens(s, window);
  if (form == kQ4Form) return s->dtype == KV_F32 ? INT_MAX : 24;
  if (s->dtype == KV_F32) return form == kOwnForm ? 0 : seen <= 1024 ? 64 : INT_MAX;
  const bool is_short = seen <= 4096;
  return form != kOwnForm ? (is_short ? 24 : 16) : (is_short ? 16 : 8);
}
// The 4-bit cache's kernel for few rows: above so many tokens that a row may see, eight
// warps a CTA, which leaves half as many parts to join; up to it four, between which short
// units divide better.  (us, four / eight, 8 kv heads, 8 rows: 8 x 64k 105 / 102, 4 x 32k 38 /
// 34, 16 x 8k 33 / 33, 4 x 8k 24 / 20, 32 x 4k 32 / 32, 4 x 4k 21 / 16, 64 x 2k 32 / 35, 16 x 2k
// 18.3 / 18.9, 4 x 700 9.4 / 10; 32 kv heads, one row, 64 x 2k 107 / 128, 8 x 16k 102 / 102.)
#ifndef KVS_Q4_EIGHT_WARPS
#define KVS_Q4_EIGHT_WARPS 4000
#endif
// fp32: up to this many packed rows K and V go straight to registers, in units of
// 4 or 8 rows; above, through shared memory in units of 64.  (4 x 8k tokens, 8 kv
// heads, us, units of 8 / of 64: 12 rows 73 / 175, 24 rows 111 / 176, 32 rows 131 /
// 176; about even at 48.)
#ifndef KVS_F32_FEW_ROWS
#define KVS_F32_FEW_ROWS 40
#endif
struct ChunkPlan {
  bool mma = false;   // tensor cores (16-bit data)
  bool q8 = false;    // the kernel reads the 8-bit cache itself
  bool q4 = false;    // the kernel reads the 4-bit cache itself
  bool few = false;   // the kernel for few rows
  bool eight = false; // whose CTAs have eight warps, not four (4-bit cache)
  bool stage = false; // K/V pass through the workspace, in the shape's type
  bool renumber = false;  // the staged pages have a block table of their own
  long long stage_pages = 0;
  int rows = 64;      // packed rows per unit
  int tile = 64;      // tokens per KV tile
  int row_tile = 0;   // tensor cores: packed rows per Q tile (a unit is one, or two when wide)
  ChunkForm form = kPair;
  // Tiles that a unit counts beyond its own: its start and its end.  (us at 0 / 1 / 2:
  // 32 prompts of 2000, 32/8 heads, kWide 405 / 385 / 374; of 512, kSolo 75 / 68 / 68;
  // fp32 over 8 bits, 32 x 300 tokens 17.6 / 16.2 / 16.0; one token, 4 x 700, 8 bits 9.7
  // / 10.1 / 10.2.)
  int unit_cost = 1;
  double most_tiles = 0;  // an upper bound of the call's (unit, KV tile) pairs
  int ctas = 1;
  bool many_parts = false;  // units are shared by 16 CTAs and more
  int slot_rows = 1;  // rows of a partial result
  size_t off_meta = 0, off_ml = 0, off_o = 0, off_table = 0, off_k = 0, off_v = 0;
  size_t total = 0;
};

// Everything here follows from the shape and the host's bounds; the lengths
// are known on the device only.  coarse: the kernels with the largest units, whatever
// they cost.
ChunkPlan chunk_plan(const kv_shape *s, const kv_chunk *c, CacheForm form, bool coarse) {
  ChunkPlan pl;
  const bool q8 = form == kQ8Form, q4 = form == kQ4Form;
  const int dev = current_device();
  const int sms = dev >= 0 ? sm_count(dev) : 152;
  const int G = s->num_q_heads / s->num_kv_heads;
  const long long packed = (long long)std::min(c->max_q_len, c->total_q) * G;
  pl.mma = s->dtype != KV_F32;
  const bool hbm = s->kv_loc == KV_LOC_HBM;
  int per_sm = 2;
  pl.q8 = q8 && hbm;
  pl.q4 = q4 && hbm;
  pl.few = !coarse &&
           packed <= few_rows_limit(s, c->window, pl.q8 ? kQ8Form : pl.q4 ? kQ4Form : kOwnForm);
  if (pl.few) {
    pl.stage = !hbm;
    pl.eight = pl.q4 && s->dtype != KV_F32 && seen_tokens(s, c->window) > KVS_Q4_EIGHT_WARPS;
    const FewShape sh = pl.q4 ? chunk_q4_shape(s->dtype, pl.eight) : chunk_few_shape(s->dtype, pl.q8);
    pl.rows = sh.rows;
    pl.tile = sh.tile;
    per_sm = sh.per_sm;
  } else if (pl.mma) {
    pl.tile = kChunkTile;
    // a Q tile holds whole tokens, for the TMA unit, where a token's heads fit
    pl.row_tile = G <= 128 ? 128 / G * G : 128;
    const long long seen = seen_tokens(s, c->window);
    const bool many = packed > pl.row_tile, wide = coarse && many;
    pl.q8 &= packed <= KVS_Q8_DIRECT_ROWS && !wide;
    pl.q4 &= packed <= KVS_Q4_DIRECT_ROWS && !wide;
    pl.stage = (q8 && !pl.q8) || (q4 && !pl.q4) || !hbm;
    pl.form = pl.q8                                                        ? kPair8
              : pl.q4                                                      ? kPair4
              : seen <= (many ? KVS_SOLO_TOKENS : KVS_SOLO_FEW) && !wide ? kSolo
              : many                                                       ? kWide
                                                                           : kPair;
    pl.rows = pl.row_tile * (pl.form == kWide ? 2 : 1);
    per_sm = pl.form == kSolo ? 2 : 1;
    if (pl.form != kSolo) pl.unit_cost = 2;
  } else {
    pl.stage = q4;  // (from host memory, or coarse: else it is for the kernel above)
    // few rows in units of 4 or 8, also while units of 64 would not fill the GPU
    const double units64 = std::min((double)s->batch * ((packed + 63) / 64),
                                    (double)c->total_q * G / 64 + s->batch);
    const bool fills = units64 * s->num_kv_heads *
                           (((double)s->max_pages_per_seq * s->page_size + pl.tile - 1) / pl.tile) >=
                       per_sm * (double)sms;
    pl.rows = coarse ? 64 : packed <= 4 ? 4 : packed <= KVS_F32_FEW_ROWS || !fills ? 8 : 64;
    if (pl.rows == 8) per_sm = 1;  // resident CTAs of its kernel (registers)
  }
  // units of all sequences: full ones and one more each; no more CTAs than
  // there can be tiles
  const double units = std::min((double)s->batch * ((packed + pl.rows - 1) / pl.rows),
                                (double)c->total_q * G / pl.rows + s->batch);
  const long long tiles = ((long long)s->max_pages_per_seq * s->page_size + pl.tile - 1) / pl.tile;
  pl.most_tiles = units * s->num_kv_heads * (tiles + pl.unit_cost);
  pl.ctas = (int)std::min<double>((double)per_sm * sms, std::max(1.0, pl.most_tiles));
  pl.many_parts = pl.ctas >= 16 * units * s->num_kv_heads;
  pl.slot_rows = (int)std::min<long long>(pl.rows, packed);
  size_t off = align256((size_t)pl.ctas * 32);
  pl.off_ml = off;
  off = align256(off + (size_t)2 * pl.ctas * pl.slot_rows * 8);
  pl.off_o = off;
  off = align256(off + (size_t)2 * pl.ctas * pl.slot_rows * kHeadDim * 4);
  if (pl.stage) {
    // staged under the cache's own page numbers, or, where that takes less,
    // under the rows of the block table
    const long long rows = (long long)s->batch * s->max_pages_per_seq;
    pl.renumber = rows < s->num_phys_pages;
    pl.stage_pages = pl.renumber ? rows : s->num_phys_pages;
    const size_t page = (size_t)s->num_kv_heads * s->page_size * kHeadDim * elem_bytes(s->dtype);
    pl.off_table = off;
    if (pl.renumber) off = align256(off + (size_t)rows * 4);
    pl.off_k = off;
    off = align256(off + (size_t)pl.stage_pages * page);
    pl.off_v = off;
    off = align256(off + (size_t)pl.stage_pages * page);
  }
  pl.total = off;
  return pl;
}

// The kernels count tiles and the staging's blocks in int32, and index the staged
// cache's rows as a cache's own.
bool plan_fits(const kv_shape *s, const ChunkPlan &pl) {
  if (pl.most_tiles > INT_MAX) return false;
  return !pl.stage ||
         (pl.stage_pages <= INT_MAX / ((long long)s->num_kv_heads * s->page_size) &&
          q8_grid_fits(s->batch, s->max_pages_per_seq, s->page_size, s->num_kv_heads));
}

// The plan of a call: the fastest, or, where its units and tiles do not count in int32 (units
// of 8 rows: fp32 over the 4-bit cache, one prompt of 131072 tokens with 64/8 heads), the
// coarsest.
ChunkPlan make_chunk_plan(const kv_shape *s, const kv_chunk *c, CacheForm form) {
  const ChunkPlan pl = chunk_plan(s, c, form, false);
  if (plan_fits(s, pl)) return pl;
  return chunk_plan(s, c, form, true);
}

// A tensor map of rows of 128 channels under the 128-byte swizzle.
struct MapShape {
  int type;              // CUtensorMapDataType
  const void *base;
  long long rows;        // pages * Hkv * ps, or tokens of q
  int heads, box, box2;  // heads: 0 for pages; box: rows, or heads and tokens (box2)
};
int encode_map(const MapShape &k, CUtensorMap *map) {
  auto fn = encode_fn();
  if (!fn) return KV_ERR_CUDA;
  const bool codes = k.type == CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const cuuint64_t row = (cuuint64_t)kHeadDim * (codes ? 1 : 2);
  const cuuint32_t across = codes ? 128 : 64;  // 128 bytes
  const cuuint32_t estr[3] = {1, 1, 1};
  cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)k.rows, 0}, strides[2] = {row, 0};
  cuuint32_t box[3] = {across, (cuuint32_t)k.box, 0};
  if (k.heads) {  // q: [tokens][heads][128]
    dims[1] = (cuuint64_t)k.heads;
    dims[2] = (cuuint64_t)k.rows;
    strides[1] = row * k.heads;
    box[2] = (cuuint32_t)k.box2;
  }
  const CUresult r = fn(map, (CUtensorMapDataType)k.type, k.heads ? 3 : 2,
                        const_cast<void *>(k.base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? KV_OK : KV_ERR_CUDA;
}

int type16(const kv_shape *s) {
  return s->dtype == KV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}
// Pages as rows [pages * Hkv * ps][128]: a box is 128 bytes, 64 channels of 16-bit
// data or all 128 of codes, of a page's tokens that fall into one KV tile.
int page_map(const kv_shape *s, bool codes, int tile, const void *base, long long pages,
             CUtensorMap *map) {
  return encode_map(MapShape{codes ? (int)CU_TENSOR_MAP_DATA_TYPE_UINT8 : type16(s), base,
                             pages * s->num_kv_heads * s->page_size, 0,
                             std::min(s->page_size, tile), 0},
                    map);
}
// q: a box is 64 channels of the G heads of row_tile / G tokens.
int q_map(const kv_shape *s, const kv_chunk *c, const void *q, int row_tile,
          CUtensorMap *map) {
  const int G = s->num_q_heads / s->num_kv_heads;
  return encode_map(MapShape{type16(s), q, c->total_q, s->num_q_heads, G, row_tile / G}, map);
}

size_t chunk_bytes(const kv_shape *s, const kv_chunk *c, CacheForm form) {
  if (check_shape(s) != KV_OK || check_chunk(s, c) != KV_OK) return 0;
  const ChunkPlan pl = make_chunk_plan(s, c, form);
  return plan_fits(s, pl) ? pl.total : 0;
}

int chunk_common(const kv_shape *s, const kv_chunk *c, const void *q, const void *k_cache,
                 const void *v_cache, const kv_q8_cache *q8, const kv_q4_cache *q4, CacheForm form,
                 const int32_t *bt, const int32_t *ctx, float scale, void *out, void *workspace,
                 size_t ws_bytes, void *stream) {
  int rc = check_shape(s);
  if (rc) return rc;
  if ((rc = check_chunk(s, c)) != KV_OK) return rc;
  if (!al16(q) || !al16(out) || !al4(bt) || !al4(ctx) || !std::isfinite(scale))
    return KV_ERR_INVALID_ARG;
  const ChunkPlan pl = make_chunk_plan(s, c, form);
  if (!plan_fits(s, pl)) return KV_ERR_UNSUPPORTED;
  const int dev = current_device();
  if (dev < 0) return KV_ERR_CUDA;
  ChunkArgs a = {};
  if (form == kQ4Form) {
    kv_q4_cache d;
    if ((rc = resolve_q4(s, q4, &d)) != KV_OK) return rc;
    a.k = d.k_codes;
    a.v = d.v_codes;
    a.k_scale = d.k_power;
    a.v_scale = d.v_power;
    a.k_group = d.k_scale;
    a.v_group = d.v_scale;
  } else if (form == kQ8Form) {
    kv_q8_cache d;
    if ((rc = resolve_q8(s, q8, &d)) != KV_OK) return rc;
    a.k = d.k_codes;
    a.v = d.v_codes;
    a.k_scale = d.k_scale;
    a.v_scale = d.v_scale;
  } else {
    if ((rc = resolve_kv(s, k_cache, &a.k)) != KV_OK) return rc;
    if ((rc = resolve_kv(s, v_cache, &a.v)) != KV_OK) return rc;
  }
  if (!al16(workspace) || ws_bytes < pl.total) return KV_ERR_WORKSPACE;
  int *status = status_ptr(dev);
  if (!status) return KV_ERR_CUDA;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.q = q;
  a.q_start = c->q_start;
  a.bt = bt;
  a.ctx = ctx;
  a.out = out;
  a.part_o = reinterpret_cast<float *>(ws + pl.off_o);
  a.part_ml = reinterpret_cast<float *>(ws + pl.off_ml);
  a.meta = reinterpret_cast<int4 *>(ws + pl.off_meta);
  a.status = status;
  a.nphys = s->num_phys_pages;
  a.B = s->batch;
  a.Hq = s->num_q_heads;
  a.Hkv = s->num_kv_heads;
  a.G = s->num_q_heads / s->num_kv_heads;
  a.ps = s->page_size;
  a.maxP = s->max_pages_per_seq;
  a.total_q = c->total_q;
  a.max_q_len = c->max_q_len;
  // a window as wide as the longest row is no window
  a.window = c->window >= (long long)a.maxP * a.ps ? 0 : c->window;
  a.slot_rows = pl.slot_rows;
  a.unit_cost = pl.unit_cost;
  a.by_g = Divisor::of(a.G);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.wait_limit_ns = wait_limit_ns();
  a.debug_skip_tile = debug_skip_page() < 0 ? -1 : debug_skip_page() / (pl.tile / kTileTokens);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  long long pages = s->num_phys_pages;
  if (pl.stage) {
    int32_t *table = pl.renumber ? reinterpret_cast<int32_t *>(ws + pl.off_table) : nullptr;
    if (launch_chunk_stage(s->dtype, form, a, ws + pl.off_k, ws + pl.off_v, table, st) !=
        cudaSuccess)
      return KV_ERR_CUDA;
    a.k = ws + pl.off_k;
    a.v = ws + pl.off_v;
    if (table) a.bt = table;
    a.nphys = pages = pl.stage_pages;
  }
  CUtensorMap tq = {}, tk = {}, tv = {};
  if ((pl.few && !pl.q4) || (pl.mma && !pl.few && !pl.q8 && !pl.q4)) {
    if ((rc = page_map(s, pl.q8, pl.tile, a.k, pages, &tk)) != KV_OK) return rc;
    if ((rc = page_map(s, pl.q8, pl.tile, a.v, pages, &tv)) != KV_OK) return rc;
  }
  if (pl.few && pl.q4) {
    e = launch_chunk_q4(s->dtype, pl.eight, a, pl.ctas, st);
  } else if (pl.few) {
    e = launch_chunk_few(s->dtype, pl.q8, a, tk, tv, pl.ctas, st);
  } else if (pl.mma) {
    a.row_tile = pl.row_tile;
    // a scale that is not positive is applied to Q as it is loaded
    a.q_tma = a.G <= pl.row_tile && pl.row_tile % a.G == 0 && a.scale_log2 > 0.f;
    if (a.q_tma && (rc = q_map(s, c, q, pl.row_tile, &tq)) != KV_OK) return rc;
    e = launch_chunk_mma(s->dtype, pl.form, a, tq, tk, tv, pl.ctas, st);
  } else {
    e = launch_chunk_core(a, form == kQ8Form, pl.rows, pl.ctas, st);
  }
  if (e == cudaSuccess) e = launch_chunk_combine(s->dtype, a, pl.ctas, pl.many_parts, st);
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

int check_append(const kv_shape *s, const kv_chunk *c, const void *k_new, const void *v_new,
                 const int32_t *bt, const int32_t *ctx, const int32_t *ctx_out) {
  int rc = check_shape(s);
  if (rc) return rc;
  if ((rc = check_chunk(s, c)) != KV_OK) return rc;
  if (!al16(k_new) || !al16(v_new) || !al4(bt) || !al4(ctx) || (ctx_out && !al4(ctx_out)))
    return KV_ERR_INVALID_ARG;
  // the same array or one apart, not one that overlaps
  if (ctx_out && ctx_out != ctx && ctx_out < ctx + s->batch && ctx < ctx_out + s->batch)
    return KV_ERR_INVALID_ARG;
  return KV_OK;
}

int check_read(const kv_shape *s, const int32_t *bt, const int32_t *ctx, const int32_t *out_table,
               int64_t out_pages, const void *k_out, const void *v_out) {
  const int rc = check_shape(s);
  if (rc) return rc;
  if (!al16(k_out) || !al16(v_out) || !al4(bt) || !al4(ctx) || !al4(out_table) || out_pages < 1)
    return KV_ERR_INVALID_ARG;
  if (out_pages > INT_MAX / ((long long)s->num_kv_heads * s->page_size) ||
      !q8_grid_fits(s->batch, s->max_pages_per_seq, s->page_size, s->num_kv_heads))
    return KV_ERR_UNSUPPORTED;
  return KV_OK;
}
// The pages read back are in device memory whatever kv_loc says.
int resolve_read(const kv_shape *s, void **k_out, void **v_out) {
  kv_shape hbm = *s;
  hbm.kv_loc = KV_LOC_HBM;
  for (void **p : {k_out, v_out}) {
    const void *at = nullptr;
    const int rc = resolve_kv(&hbm, *p, &at);
    if (rc != KV_OK) return rc;
    *p = const_cast<void *>(at);
  }
  return KV_OK;
}

int check_rope(const kv_rope_plan *r) {
  if (!r || !r->freq || ((uintptr_t)r->freq & 7u) || ((uintptr_t)r->positions & 3u) ||
      (r->interleaved != 0 && r->interleaved != 1) || !std::isfinite(r->scale) || r->reserved != 0)
    return KV_ERR_INVALID_ARG;
  return r->rotary_dim >= 8 && r->rotary_dim <= kHeadDim && r->rotary_dim % 8 == 0
             ? KV_OK
             : KV_ERR_UNSUPPORTED;
}
// The bytes of a [total_q][heads][d] array.
struct Rows {
  const uint8_t *at;
  size_t bytes;
};
Rows rows_of(const kv_shape *s, const kv_chunk *c, const void *p, bool q) {
  return Rows{static_cast<const uint8_t *>(p), (size_t)c->total_q * kHeadDim * elem_bytes(s->dtype) *
                                                   (q ? s->num_q_heads : s->num_kv_heads)};
}
// Whether arrays are aligned, and no output meets another array in part or out of place:
// the first `in_out` pairs of rows are an input and its output, which may be one array.
bool rows_apart(const Rows *r, int n, int in_out) {
  for (int i = 0; i < n; ++i) {
    if (r[i].at && !al16(r[i].at)) return false;
    for (int j = 0; j < i; ++j) {
      const bool out_i = i < 2 * in_out && (i & 1), out_j = j < 2 * in_out && (j & 1);
      if (!r[i].at || !r[j].at || (!out_i && !out_j)) continue;
      if (out_i && j == i - 1 && r[i].at == r[j].at) continue;
      if (r[i].at < r[j].at + r[j].bytes && r[j].at < r[i].at + r[i].bytes) return false;
    }
  }
  return true;
}

// Whether what an append writes, the cache and its index (may be null), meets neither its rows
// nor itself.  (k, v: as the device sees them, like the rows.)
bool cache_apart(const kv_shape *s, const void *k, const void *v, const void *mm, const Rows *rows,
                 int n) {
  const size_t head = (size_t)s->num_phys_pages * s->num_kv_heads * kHeadDim * elem_bytes(s->dtype);
  const Rows out[3] = {{static_cast<const uint8_t *>(k), head * s->page_size},
                       {static_cast<const uint8_t *>(v), head * s->page_size},
                       {static_cast<const uint8_t *>(mm), head * 2}};
  const auto meet = [](const Rows &x, const Rows &y) {
    return x.at && y.at && x.at < y.at + y.bytes && y.at < x.at + x.bytes;
  };
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return false;
    for (int j = 0; j < n; ++j)
      if (meet(out[i], rows[j])) return false;
  }
  return true;
}

}  // namespace

extern "C" {

size_t kv_chunk_workspace_bytes(const kv_shape *shape, const kv_chunk *chunk) {
  return chunk_bytes(shape, chunk, kOwnForm);
}

size_t kv_q8_chunk_workspace_bytes(const kv_shape *shape, const kv_chunk *chunk) {
  return chunk_bytes(shape, chunk, kQ8Form);
}

int kv_chunk_attn(const kv_shape *shape, const kv_chunk *chunk, const void *q,
                  const void *k_cache, const void *v_cache, const int32_t *block_table,
                  const int32_t *context_lens, float scale, void *out, void *workspace,
                  size_t workspace_bytes, void *stream) {
  KV_API_RANGE();
  return chunk_common(shape, chunk, q, k_cache, v_cache, nullptr, nullptr, kOwnForm, block_table,
                      context_lens, scale, out, workspace, workspace_bytes, stream);
}

int kv_q8_chunk_attn(const kv_shape *shape, const kv_chunk *chunk, const void *q,
                     const kv_q8_cache *cache, const int32_t *block_table,
                     const int32_t *context_lens, float scale, void *out, void *workspace,
                     size_t workspace_bytes, void *stream) {
  KV_API_RANGE();
  return chunk_common(shape, chunk, q, nullptr, nullptr, cache, nullptr, kQ8Form, block_table,
                      context_lens, scale, out, workspace, workspace_bytes, stream);
}

int kv_q8_append(const kv_shape *shape, const kv_chunk *chunk, const void *k_new,
                 const void *v_new, const kv_q8_cache *cache, const int32_t *block_table,
                 const int32_t *context_lens, int32_t *context_lens_out, void *stream) {
  KV_API_RANGE();
  int rc = check_append(shape, chunk, k_new, v_new, block_table, context_lens, context_lens_out);
  if (rc) return rc;
  const int dev = current_device();
  if (dev < 0) return KV_ERR_CUDA;
  kv_q8_cache d;
  if ((rc = resolve_q8(shape, cache, &d)) != KV_OK) return rc;
  int *status = status_ptr(dev);
  if (!status) return KV_ERR_CUDA;
  const cudaError_t e = launch_q8_append(
      shape->dtype, k_new, v_new, d, chunk->q_start, block_table, context_lens, context_lens_out,
      shape->batch, shape->num_kv_heads, shape->page_size, shape->max_pages_per_seq,
      shape->num_phys_pages, chunk->total_q, chunk->max_q_len, status,
      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

int kv_q8_read(const kv_shape *shape, const kv_q8_cache *cache, const int32_t *block_table,
               const int32_t *context_lens, const int32_t *out_table, int64_t out_pages,
               void *k_out, void *v_out, void *stream) {
  KV_API_RANGE();
  int rc = check_read(shape, block_table, context_lens, out_table, out_pages, k_out, v_out);
  if (rc) return rc;
  const int dev = current_device();
  if (dev < 0) return KV_ERR_CUDA;
  kv_q8_cache d;
  if ((rc = resolve_q8(shape, cache, &d)) != KV_OK) return rc;
  if ((rc = resolve_read(shape, &k_out, &v_out)) != KV_OK) return rc;
  int *status = status_ptr(dev);
  if (!status) return KV_ERR_CUDA;
  const cudaError_t e = launch_q8_read(
      shape->dtype, d, block_table, context_lens, out_table, out_pages, k_out, v_out,
      shape->batch, shape->num_kv_heads, shape->page_size, shape->max_pages_per_seq,
      shape->num_phys_pages, status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

int kv_q4_append(const kv_shape *shape, const kv_chunk *chunk, const void *k_new,
                 const void *v_new, const kv_q4_cache *cache, const int32_t *block_table,
                 const int32_t *context_lens, int32_t *context_lens_out, void *stream) {
  KV_API_RANGE();
  int rc = check_append(shape, chunk, k_new, v_new, block_table, context_lens, context_lens_out);
  if (rc) return rc;
  const int dev = current_device();
  if (dev < 0) return KV_ERR_CUDA;
  kv_q4_cache d;
  if ((rc = resolve_q4(shape, cache, &d)) != KV_OK) return rc;
  int *status = status_ptr(dev);
  if (!status) return KV_ERR_CUDA;
  const cudaError_t e = launch_q4_append(
      shape->dtype, k_new, v_new, d, chunk->q_start, block_table, context_lens, context_lens_out,
      shape->batch, shape->num_kv_heads, shape->page_size, shape->max_pages_per_seq,
      shape->num_phys_pages, chunk->total_q, chunk->max_q_len, status,
      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

int kv_q4_read(const kv_shape *shape, const kv_q4_cache *cache, const int32_t *block_table,
               const int32_t *context_lens, const int32_t *out_table, int64_t out_pages,
               void *k_out, void *v_out, void *stream) {
  KV_API_RANGE();
  int rc = check_read(shape, block_table, context_lens, out_table, out_pages, k_out, v_out);
  if (rc) return rc;
  const int dev = current_device();
  if (dev < 0) return KV_ERR_CUDA;
  kv_q4_cache d;
  if ((rc = resolve_q4(shape, cache, &d)) != KV_OK) return rc;
  if ((rc = resolve_read(shape, &k_out, &v_out)) != KV_OK) return rc;
  int *status = status_ptr(dev);
  if (!status) return KV_ERR_CUDA;
  const cudaError_t e = launch_q4_read(
      shape->dtype, d, block_table, context_lens, out_table, out_pages, k_out, v_out,
      shape->batch, shape->num_kv_heads, shape->page_size, shape->max_pages_per_seq,
      shape->num_phys_pages, status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

size_t kv_q4_chunk_workspace_bytes(const kv_shape *shape, const kv_chunk *chunk) {
  return chunk_bytes(shape, chunk, kQ4Form);
}

int kv_q4_chunk_attn(const kv_shape *shape, const kv_chunk *chunk, const void *q,
                     const kv_q4_cache *cache, const int32_t *block_table,
                     const int32_t *context_lens, float scale, void *out, void *workspace,
                     size_t workspace_bytes, void *stream) {
  KV_API_RANGE();
  return chunk_common(shape, chunk, q, nullptr, nullptr, nullptr, cache, kQ4Form, block_table,
                      context_lens, scale, out, workspace, workspace_bytes, stream);
}

int kv_rope(const kv_shape *shape, const kv_chunk *chunk, const kv_rope_plan *rope, const void *q,
            void *q_out, const void *k, void *k_out, const int32_t *context_lens, void *stream) {
  KV_API_RANGE();
  int rc = check_shape(shape);
  if (rc) return rc;
  if ((rc = check_chunk(shape, chunk)) != KV_OK) return rc;
  if ((rc = check_rope(rope)) != KV_OK) return rc;
  if ((!q && !k) || !q != !q_out || !k != !k_out) return KV_ERR_INVALID_ARG;
  if (context_lens ? !al4(context_lens) : !rope->positions) return KV_ERR_INVALID_ARG;
  const Rows rows[4] = {rows_of(shape, chunk, q, true), rows_of(shape, chunk, q_out, true),
                        rows_of(shape, chunk, k, false), rows_of(shape, chunk, k_out, false)};
  if (!rows_apart(rows, 4, 2)) return KV_ERR_INVALID_ARG;
  int blocks;
  if (!rope_grid(shape, chunk, false, 16, &blocks)) return KV_ERR_UNSUPPORTED;
  const int dev = current_device();
  if (dev < 0) return KV_ERR_CUDA;
  int *status = status_ptr(dev);
  if (!status) return KV_ERR_CUDA;
  // (lengths that do not give the positions are not read)
  const cudaError_t e =
      launch_rope(shape, chunk, rope, q, q_out, k, k_out, nullptr, nullptr, nullptr,
                  rope->positions ? nullptr : context_lens, nullptr, nullptr, status,
                  static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

int kv_rope_append(const kv_shape *shape, const kv_chunk *chunk, const kv_rope_plan *rope,
                   const void *q, void *q_out, const void *k_new, const void *v_new, void *k_cache,
                   void *v_cache, const int32_t *block_table, const int32_t *context_lens,
                   int32_t *context_lens_out, void *minmax, void *stream) {
  KV_API_RANGE();
  int rc = check_append(shape, chunk, k_new, v_new, block_table, context_lens, context_lens_out);
  if (rc) return rc;
  if (rope && (rc = check_rope(rope)) != KV_OK) return rc;
  if (!q != !q_out || (q && !rope) || (minmax && !al16(minmax))) return KV_ERR_INVALID_ARG;
  const Rows rows[4] = {rows_of(shape, chunk, q, true), rows_of(shape, chunk, q_out, true),
                        rows_of(shape, chunk, k_new, false), rows_of(shape, chunk, v_new, false)};
  if (!rows_apart(rows, 4, 1)) return KV_ERR_INVALID_ARG;
  int blocks;
  if (!rope_grid(shape, chunk, true, minmax ? shape->page_size : 16, &blocks))
    return KV_ERR_UNSUPPORTED;
  const int dev = current_device();
  if (dev < 0) return KV_ERR_CUDA;
  const void *k = nullptr, *v = nullptr;
  if ((rc = resolve_kv(shape, k_cache, &k)) != KV_OK) return rc;
  if ((rc = resolve_kv(shape, v_cache, &v)) != KV_OK) return rc;
  if (!cache_apart(shape, k, v, minmax, rows, 4)) return KV_ERR_INVALID_ARG;
  int *status = status_ptr(dev);
  if (!status) return KV_ERR_CUDA;
  const cudaError_t e = launch_rope(shape, chunk, rope, q, q_out, k_new, const_cast<void *>(k), v_new,
                                    const_cast<void *>(v), block_table, context_lens,
                                    context_lens_out, minmax, status,
                                    static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

}  // extern "C"
