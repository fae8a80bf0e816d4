// kv_chunk.cuh -- attention of a chunk of new tokens over a paged cache: what
// its kernels share, above all how the work is cut.
//
// What it computes, for row i of sequence b's n_b new tokens (token t = len_b
// - n_b + i) and query head h:
//   out = sum_j softmax_j(scale * q . k_j) v_j,   max(0, t - window + 1) <= j <= t
//
// Work.  The G query heads of a kv head read the same K and V, so their rows
// are packed: packed row r = i * G + g is token i, head kvh * G + g.  A unit
// is `rows` consecutive packed rows of one (sequence, kv head); it meets the
// KV tiles [tile_lo, tile_hi) its rows can see, one at least.  All units' tiles, and a
// cost of a tile or two per unit, laid end to end (sequence, kv head, row block;
// lengths differ, so the total is known on the device only) are cut into equal
// shares, one per CTA, as many CTAs as are resident.  A
// share is a list of segments: the end of one unit, whole units, the start of
// another.  A unit within one share is written to out; the others leave
// partial results (at most two per CTA, so the workspace does not grow with
// the batch) that the combine kernel joins.  Ragged batches, one long
// sequence and many short ones are balanced by the same rule to one tile.
#pragma once

#include <climits>

#include "kv_internal.cuh"
#include "kv_q8.cuh"

namespace kvs {

constexpr int kChunkTile = 128;  // tokens per KV tile of the tensor-core kernels

struct ChunkArgs {
  const void *q;
  const void *k, *v;                // K and V (8-bit: the codes)
  const uint8_t *k_scale, *v_scale; // 8-bit only
  const int32_t *q_start, *bt, *ctx;
  void *out;
  float *part_o;    // [2 * ctas][slot_rows][d]
  float *part_ml;   // [2 * ctas][slot_rows][2]: log2-domain maximum, sum
  int4 *meta;       // [ctas][2]: the unit whose first tile lies in the CTA's share and whose last does not
  int *status;
  long long nphys;
  int B, Hq, Hkv, G, ps, maxP, total_q, max_q_len, window;
  int slot_rows;
  Divisor by_g;      // packed row / G
  int unit_cost;     // tiles that a unit counts beyond its own when the work is cut
  int row_tile;      // tensor cores: packed rows per Q tile
  int q_tma;         // tensor cores: Q tiles are whole tokens, copied by the TMA unit
  float scale_log2;  // scale * log2(e)
  unsigned long long wait_limit_ns;
  int debug_skip_tile;  // >= 0: the producer never fills that tile of a share (timeout test)
};

// the token of a packed row (>= 0)
__device__ __forceinline__ int token_of(const ChunkArgs &a, int row) { return a.by_g(row); }

// where packed row `row` of kv head kvh lies in q and out, rows of its sequence from q0
__device__ __forceinline__ long long row_offset(const ChunkArgs &a, int q0, int kvh, int row) {
  const int i = token_of(a, row);
  return ((long long)(q0 + i) * a.Hq + kvh * a.G + row - i * a.G) * kHeadDim;
}

// One sequence of the call; n = 0 when it has no rows or is skipped.
struct ChunkSeq {
  int q0, n, len;
};
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkArgs &a, int b, bool flag) {
  const int q0 = a.q_start[b], q1 = a.q_start[b + 1], len = a.ctx[b];
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.total_q && q1 - q0 <= a.max_q_len && len >= 0 &&
                  (long long)len <= (long long)a.maxP * a.ps;
  if (!ok && flag) flag_error(a.status, KV_ERR_BOUNDS);
  return ChunkSeq{q0, ok ? q1 - q0 : 0, len};
}

// KV tiles [lo, hi) of the unit of packed rows [r0, r0 + nrows): what its
// rows can see, and one tile where they see nothing (it writes the zeros).
struct TileRange {
  int lo, hi;
};
__device__ __forceinline__ TileRange unit_tiles(const ChunkArgs &a, const ChunkSeq &s, int r0,
                                                int nrows, int tile) {
  const int t_first = s.len - s.n + token_of(a, r0);
  const int t_last = s.len - s.n + token_of(a, r0 + nrows - 1);
  if (t_last < 0) return TileRange{0, 1};
  // (t_first >= -1 here: a window may be as large as an int32)
  const int lo = a.window > 0 ? max(0, max(t_first, -1) - a.window + 1) : 0;
  return TileRange{lo / tile, t_last / tile + 1};
}

// One segment of a CTA's share.
struct ChunkSeg {
  int b, kvh, r0, nrows;  // unit: packed rows [r0, r0 + nrows) of (b, kvh)
  int q0, n, len;         // its sequence
  int tile_lo, tile_hi;   // the KV tiles of this segment
  int parts;              // bit 0: it holds the unit's first tile, bit 1: its last
  int t_first, t_last;    // tokens of the unit's first and last row
  // KV tiles in which some row does not see some token, or that end behind the
  // sequence inside a page: those >= edge_from and those <= edge_upto
  int edge_from, edge_upto;
  int half_hi;            // end of the tiles that the first half of a full unit's rows sees
  __device__ __forceinline__ bool first() const { return parts & 1; }
  __device__ __forceinline__ bool whole() const { return parts == 3; }
};
// The first token that some row of the segment's unit sees.  A page out of range before
// it is nobody's: the caller may have given it back.  (t_first >= -1, as in unit_tiles)
__device__ __forceinline__ int seen_from(const ChunkArgs &a, const ChunkSeg &g) {
  return a.window > 0 ? max(g.t_first, -1) - a.window + 1 : 0;
}

// A CTA's share, kSegs segments of it listed at a time.
template <int kSegs> struct ChunkShare {
  // (the host refuses calls whose tiles might not fit int32)
  int per, extra;          // share: what it counts; the first `extra` shares hold one more
  int hi;                  // end of this CTA's share in the units laid end to end
  int b, kvh, r0, off;     // walk: the next unit, and how much of it is passed
  int left;                // of the share, not listed yet
  int nseg;
  ChunkSeg seg[kSegs];
};

__device__ __forceinline__ int packed_rows(const ChunkArgs &a, const ChunkSeq &s) {
  return s.n * a.G;  // checked on the host against int32 (max_q_len * G)
}
// What the unit of packed rows from r0 on counts when the work is cut: its tiles,
// and unit_cost.  (Its tiles come first: a share that ends among the rest ends
// behind the unit, whole.)
__device__ __forceinline__ int unit_counts(const ChunkArgs &a, const ChunkSeq &s, int r0, int R,
                                           int rows, int tile) {
  const TileRange t = unit_tiles(a, s, r0, min(rows, R - r0), tile);
  return t.hi - t.lo + a.unit_cost;
}
// all row blocks of one kv head of sequence s from r0 on, every `step` rows
__device__ __forceinline__ int head_counts(const ChunkArgs &a, const ChunkSeq &s, int r0, int step,
                                           int rows, int tile) {
  const int R = packed_rows(a, s);
  int w = 0;
#pragma unroll 1
  for (; r0 < R; r0 += step) w += unit_counts(a, s, r0, R, rows, tile);
  return w;
}
__device__ __forceinline__ int scan_lanes(int w, int lane) {  // inclusive
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, w, off);
    if (lane >= off) w += x;
  }
  return w;
}

// Every thread of the CTA: the total work, this CTA's share and where it
// starts.  red: 32 ints of shared scratch.  A warp takes a sequence's row blocks
// 32 at a time where there are no more sequences than warps, else a thread does
// (2 sequences of 16 row blocks: 176 -> 169 us of a call of 1000 new tokens over 16000).
template <int kSegs>
__device__ __forceinline__ void share_init(const ChunkArgs &a, int rows, int tile,
                                           ChunkShare<kSegs> *sh, int *red) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, nw = blockDim.x >> 5;
  const bool by_warp = a.B <= nw;
  int first = 0, mine = 0;  // counts of this thread's first sequence, of all of its
  if (by_warp) {
    if (warp < a.B)
      mine = head_counts(a, chunk_seq(a, warp, blockIdx.x == 0 && lane == 0), lane * rows,
                         32 * rows, rows, tile);
  } else {
#pragma unroll 1
    for (int b = t; b < a.B; b += blockDim.x) {
      const int w = head_counts(a, chunk_seq(a, b, blockIdx.x == 0), 0, rows, rows, tile);
      if (b == t) first = w;
      mine += w;
    }
  }
  mine = __reduce_add_sync(0xFFFFFFFFu, mine);
  if (lane == 0) red[warp] = mine;
  __syncthreads();
  if (t == 0) {
    int w = 0;
#pragma unroll 1
    for (int i = 0; i < nw; ++i) w += red[i];
    w *= a.Hkv;
    const int n = gridDim.x, i = blockIdx.x;
    sh->per = w / n;
    sh->extra = w % n;
    sh->left = sh->per + (i < sh->extra ? 1 : 0);
    sh->hi = sh->per * i + min(i, sh->extra) + sh->left;
    sh->b = -1;
    sh->nseg = 0;
  }
  __syncthreads();
  if (sh->left == 0) return;
  // the sequence in which the share begins: one warp walks the sequences 32 at a
  // time, and then its row blocks
  if (warp == 0) {
    int base = 0;
    const int want = sh->hi - sh->left;
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      ChunkSeq s{0, 0, 0};
      if (b < a.B) s = chunk_seq(a, b, false);
      const int hw = by_warp   ? (b < a.B ? red[lane] : 0)
                     : b0 == 0 ? first
                               : head_counts(a, s, 0, rows, rows, tile);
      const int inc = scan_lanes(hw * a.Hkv, lane), from = base + inc - hw * a.Hkv;
      const uint32_t here = __ballot_sync(0xFFFFFFFFu, want >= from && want < base + inc);
      if (here) {
        const int src = __ffs(here) - 1, head = __shfl_sync(0xFFFFFFFFu, hw, src);
        const ChunkSeq q{__shfl_sync(0xFFFFFFFFu, s.q0, src), __shfl_sync(0xFFFFFFFFu, s.n, src),
                         __shfl_sync(0xFFFFFFFFu, s.len, src)};
        int rem = want - __shfl_sync(0xFFFFFFFFu, from, src);
        const int kvh = rem / head, R = packed_rows(a, q);
        rem -= kvh * head;
        int r0 = 0;
#pragma unroll 1
        while (true) {
          const int mr = r0 + lane * rows;
          const int c = mr < R ? unit_counts(a, q, mr, R, rows, tile) : 0;
          const int ci = scan_lanes(c, lane);
          const uint32_t past = __ballot_sync(0xFFFFFFFFu, ci > rem);
          if (past) {
            const int k = __ffs(past) - 1;
            r0 += k * rows;
            rem -= __shfl_sync(0xFFFFFFFFu, ci - c, k);
            break;
          }
          if (r0 + 32 * rows >= R) break;  // (not reached: the counts add up to head)
          rem -= __shfl_sync(0xFFFFFFFFu, ci, 31);
          r0 += 32 * rows;
        }
        if (lane == 0) {
          sh->b = b0 + src;
          sh->kvh = kvh;
          sh->r0 = r0;
          sh->off = rem;
        }
        break;
      }
      base += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
  }
  __syncthreads();
}

// One thread: the next segments of the share (nseg = 0 when it is used up).
// The CTA that holds a unit's first tile but not its last records where the
// combine finds the rest: slot 2 i + 1 of CTA i (a share's last segment) for
// the first part, slot 2 j (a share's first segment) for each further part.
template <int kSegs>
__device__ __forceinline__ void share_next(const ChunkArgs &a, int rows, int tile,
                                           ChunkShare<kSegs> *sh) {
  int n = 0;
  if (sh->left > 0 && sh->b >= 0) {
    int b = sh->b, kvh = sh->kvh, r0 = sh->r0, off = sh->off;
    int left = sh->left;
    ChunkSeq s = chunk_seq(a, b, false);
    int R = packed_rows(a, s);
#pragma unroll 1
    while (n < kSegs && left > 0) {
      const int nrows = min(rows, R - r0);
      const TileRange t = unit_tiles(a, s, r0, nrows, tile);
      const int tiles = t.hi - t.lo;
      const int take = min(tiles + a.unit_cost - off, left);
      const int tile_hi = min(off + take, tiles);
      // (written over by the next one where none of the unit's tiles is in the share)
      ChunkSeg &g = sh->seg[n];
      if (off < tiles) ++n;
      g.b = b;
      g.kvh = kvh;
      g.r0 = r0;
      g.nrows = nrows;
      g.q0 = s.q0;
      g.n = s.n;
      g.len = s.len;
      g.tile_lo = t.lo + off;
      g.tile_hi = t.lo + tile_hi;
      g.parts = (off == 0 ? 1 : 0) | (tile_hi == tiles ? 2 : 0);
      g.t_first = s.len - s.n + token_of(a, r0);
      g.t_last = s.len - s.n + token_of(a, r0 + nrows - 1);
      g.edge_from = g.t_first < s.len - 1        ? max(g.t_first + 1, 0) / tile
                    : (s.len & (a.ps - 1)) != 0 ? s.len / tile
                                                : INT_MAX;
      g.edge_upto = a.window > 0 && g.t_last >= a.window ? (g.t_last - a.window) / tile : -1;
      const int t_half = s.len - s.n + token_of(a, r0 + min(nrows, rows / 2) - 1);
      g.half_hi = max(t_half, 0) / tile + 1;
      if (g.parts == 1) {
        // the CTA whose share holds the unit's last tile
        const int end = sh->hi - left + tiles - 1, big = sh->extra * (sh->per + 1);
        const int j = end < big ? end / (sh->per + 1) : sh->extra + (end - big) / sh->per;
        a.meta[2 * blockIdx.x] = make_int4(b, kvh, r0, nrows);
        a.meta[2 * blockIdx.x + 1] = make_int4(s.q0, j, 0, 0);
      }
      left -= take;
      off = 0;
      r0 += rows;
      if (r0 >= R) {
        r0 = 0;
        if (++kvh == a.Hkv) {
          kvh = 0;
          s.n = 0;
#pragma unroll 1
          while (left > 0 && ++b < a.B) {
            s = chunk_seq(a, b, false);
            if (s.n > 0) break;
          }
          R = packed_rows(a, s);
          if (R == 0) break;
        }
      }
    }
    sh->b = b;
    sh->kvh = kvh;
    sh->r0 = r0;
    sh->off = 0;
    sh->left = n > 0 && R == 0 ? 0 : left;
  }
  sh->nseg = n;
}

// partial-result slot of a segment that is not a whole unit
__device__ __forceinline__ int part_slot(const ChunkSeg &g) {
  return 2 * (int)blockIdx.x + (g.first() ? 1 : 0);
}

// visible columns [lo, hi] of a tile starting at token tile0, for token t
__device__ __forceinline__ int vis_hi(int t, int tile0) { return t - tile0; }
__device__ __forceinline__ int vis_lo(int t, int tile0, int window) {
  return window > 0 ? t - tile0 - window + 1 : 0;
}

// Infinities and NaN of V.  A channel in which a row sees some is their sum: the
// weights are positive, however small.  The products do not give that everywhere: a
// weight may have rounded to 0, and where some row does not see a token its infinities
// and NaN are kept out of the products.  So where a row's result is not finite, or
// something was kept out, the cache is read again (seldom) and the sum written over the
// channel: by the attention kernels for whole units, by the combine for the others.
// (Rows whose weights are NaN stay as they are, NaN in every channel.)
__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }
__device__ __forceinline__ bool finite(const float4 &x) {
  return finite(x.x) && finite(x.y) && finite(x.z) && finite(x.w);
}
__device__ __forceinline__ void load_n(const float *p, float (&x)[4]) {
  const float4 w = *reinterpret_cast<const float4 *>(p);
  x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
}
template <class T>
__device__ __forceinline__ void load_n(const T *p, float (&x)[4]) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  const float2 u = unpack2(w.x, T{}), v = unpack2(w.y, T{});
  x[0] = u.x; x[1] = u.y; x[2] = v.x; x[3] = v.y;
}
template <class T> __device__ __forceinline__ void load_n(const T *p, float (&x)[8]) { load8(p, x); }
// The tokens lo .. hi of KV tiles [first, end) that the row at token t sees.
struct Seen {
  int lo, hi;
};
__device__ __forceinline__ Seen seen_tokens(const ChunkArgs &a, int t, int first, int end, int tile) {
  return Seen{max(first * tile, a.window > 0 ? t - a.window + 1 : 0),
              min((end - 1) * tile + tile - 1, t)};
}
// What of `N` channels is not finite, a bit each: +infinities and NaN, -infinities and NaN.
// Their sum is an infinity where one of the two holds, NaN where both do.
struct Odd {
  uint32_t plus = 0, minus = 0;
  __device__ __forceinline__ void see(int i, float x) {
    if (!(x <= 3.402823466e38f)) plus |= 1u << i;
    if (!(x >= -3.402823466e38f)) minus |= 1u << i;
  }
  __device__ __forceinline__ bool any(int i) const { return ((plus | minus) >> i) & 1; }
  __device__ __forceinline__ float sum(int i) const {
    return __uint_as_float(!((minus >> i) & 1)  ? 0x7F800000u
                           : !((plus >> i) & 1) ? 0xFF800000u
                                                : 0x7FC00000u);
  }
};
// Of tokens lo .. hi: what is not finite in channels c .. c + N - 1.  (Eight loads in
// flight: 32k tokens take a few ms.)
template <class T, int N>
__device__ __noinline__ Odd odd_values(const ChunkArgs &a, int b, int kvh, int lo, int hi, int c) {
  Odd odd;
  for (int p0 = lo & -16; p0 <= hi; p0 += 16) {
    const int ph = a.bt[(long long)b * a.maxP + p0 / a.ps];
    if (ph < 0 || ph >= a.nphys) continue;
    const T *v = static_cast<const T *>(a.v) +
                 (((long long)ph * a.Hkv + kvh) * a.ps + (p0 & (a.ps - 1))) * kHeadDim + c;
#pragma unroll 1
    for (int j0 = 0; j0 < 16; j0 += 8) {
      float x[8][N];
#pragma unroll
      for (int j = 0; j < 8; ++j) load_n(v + (j0 + j) * kHeadDim, x[j]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (p0 + j0 + j >= lo && p0 + j0 + j <= hi)
#pragma unroll
          for (int i = 0; i < N; ++i) odd.see(i, x[j][i]);
    }
    if ((odd.plus & odd.minus) == (1u << N) - 1u) break;  // NaN stays NaN
  }
  return odd;
}

// A bounded wait of a whole warp; false once anything has timed out (the kernel
// records that at its end).  The lanes vote: a barrier that completes while another
// warp calls the kernel off may look done to some lanes and not to others, which
// must not part.  Kept short: a kernel whose roles do not fit the instruction cache
// together stalls on fetches.
struct Waiter {
  volatile int *abort;
  unsigned long long limit;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_ns();
#pragma unroll 1
    while (!__any_sync(0xFFFFFFFFu, *abort)) {
      if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
      if (global_ns() - t0 > limit) *abort = 1;
    }
    return false;
  }
};

// How long a kernel that was called off waits for its own copies and products in flight
// before its shared memory and TMEM pass to another CTA.  They end by themselves, within
// microseconds (a copy from host memory too): the limit, which the waits that ran out
// may have had far shorter, only bounds the wait for a tile that was never filled.
__device__ __forceinline__ unsigned long long drain_limit(const ChunkArgs &a) {
  return max(a.wait_limit_ns, 50'000'000ull);
}

template <int kStages> struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++s == kStages) {
      s = 0;
      ph ^= 1;
    }
  }
  __device__ __forceinline__ void next(int n) {  // n <= kStages
    s += n;
    if (s >= kStages) {
      s -= kStages;
      ph ^= 1;
    }
  }
};

}  // namespace kvs
