// kv_chunk_mma.cu -- chunk attention for 16-bit data on the tensor cores
// (tcgen05, accumulators in TMEM).  kv_chunk.cuh has the formula and how the
// work is cut into shares of segments.
//
// A CTA's warps:
//   4 or 8    one or two softmax groups, a thread per packed row
//   1         loads K and V tiles (TMA, one box per page and 64 channels)
//   1         issues the matrix products (one lane)
//   2         mend V at the edges (below); the second loads Q
//   4         (8-bit, 4-bit) expand tiles of codes into the ring's 16-bit tiles
// Per KV tile of 128 tokens and softmax group: S = Q K^T (128 x 128 x 128)
// into TMEM; the group takes its maximum and exponentials and writes the
// weights P in 16 bits over S, the type that the product takes with V's (a second
// term of P would be a second product; the sum uses the unrounded weights); O += P V.  While one group computes, the tensor
// cores work for the other, of the same CTA or of another.  TMEM: S and P of
// two groups at columns 0 and 128, O at 256 and 384; of one at 0 and at 128.
//   * kWide: a unit is 256 packed rows, 128 per group; both groups use
//     each K/V tile, which halves the reads of K and V per product.
//   * kPair: a unit is up to 128 rows; the groups take its KV tiles in
//     turn (even, odd) and join their results at the end.  For few rows per
//     sequence, where the K/V stream is the bound and each tile's chain of
//     product, softmax and product would otherwise be exposed.
//   * kSolo: a unit is up to 128 rows and a CTA has one group; two CTAs per SM.
//     For short contexts, where a unit's start and end are much of it.
//   * kPair8, kPair4: kPair over the 8-bit and the 4-bit cache, up to kv_chunk_api.cu's
//     limits of rows.
//
// What bounds it, measured on one GB300 (a copy reaches 6.68 TB/s, a large bf16
// matrix product 1.91 PFLOP/s):
//   * kWide, 2048 new tokens at the end of 32768, 32/8 heads, bf16: 676-747 us
//     from box to box, 1.43-1.58 PFLOP/s.  Products and softmax share the time: the
//     tensor pipe is active for two thirds of it, and what is left is each
//     group's chain of scores, maximum, exponentials and weights.
//   * kSolo, 32 prompts of up to 512, 32/32 heads, f16: 79 us for 41 us of bytes
//     (kWide 95).  A unit has one to four tiles, each a chain of some 2900 cycles
//     (product, maximum, exponentials, product), and 3500 more to write out, which
//     two CTAs per SM cover for one another in part.
//   * kPair, 5 new tokens over 8 x 65536, 64/8 heads, bf16: 224 us, 6.7 TB/s: the
//     K/V stream.
//   * kPair8, 4 x 32768 tokens, 8 kv heads, bf16: 69 us up to 32 rows, 78 us for
//     128, 183 us for 512.  The four converting warps (eight, which leave the
//     others fewer registers, were no faster).
//   * kPair4, the same in pages of 16 / of 64: 64 rows 76 / 64 us, 512 rows 201 /
//     170 us.  Its converters, with half the bytes but more operations a code; stores
//     that meet no bank twice, for two selections a row, were no faster (f16 2 us
//     slower, bf16 up to 5 us faster).
//
// The running maximum is moved only when a row's new maximum exceeds it by
// more than 2^8 in the weights: until then the weights may be as large as 2^8,
// which neither 16-bit type nor the fp32 sums mind, and O need not be
// rescaled.  f16 weights are kept 2^7 larger, so that weights down to 2^-21
// of the maximum keep all their bits.
//
// What a row does not see must not reach it through 0 * infinity: K needs no
// care (its scores are replaced), V does.  Slots past the sequence's end in its
// last page are zeroed in shared memory before the product.  In tiles where
// some row does not see some token, infinities and NaN of V are zeroed as
// well.  Rows that do see them get them when they are written, here and where a
// result is not finite (kv_chunk.cuh; a slow path that only such data takes).
// Pages past the end or out of range are filled with zeros by the TMA unit.
#include <type_traits>

#include "kv_chunk.cuh"
#include "kv_launch.h"
#include "kv_q4.cuh"
#include "kv_q8.cuh"
#include "kv_umma.cuh"

namespace kvs {
namespace {

constexpr int kTile = kChunkTile;
constexpr int kTileBytes = kTile * kHeadDim * 2;  // 32 KB
constexpr int kSlab = kTile * 128;                // 64 channels of a tile
constexpr float kMoveAt = 8.f;  // log2 of the largest weight before the maximum moves

// How a CTA works: kMode is a ChunkForm.
template <int kMode> struct Shape {
  static constexpr bool kHalves = kMode == kWide;  // each group has half a unit's rows
  static constexpr bool kQ4 = kMode == kPair4, kQ8 = kMode == kPair8 || kQ4;  // codes; 4 bits
  static constexpr bool kTurns = kMode == kPair || kQ8;  // the groups take tiles in turn
  static constexpr int kGroups = kMode == kSolo ? 1 : 2;
  static constexpr int kCtas = kMode == kSolo ? 2 : 1;  // per SM
  static constexpr int kThreads = kMode == kSolo ? 256 : kQ8 ? 512 : 384;
  static constexpr int kQTiles = kMode == kWide ? 2 : 1;
  static constexpr int kQRows = 128;  // of a Q tile
  static constexpr int kRows = kQTiles * kQRows;
  static constexpr int kQBytes = kQRows * kHeadDim * 2;
  static constexpr int kStages = kMode == kWide ? 5 : kMode == kSolo ? 2 : kQ8 ? 4 : 6;  // 16-bit K and V tiles
  static constexpr int kRaw = kQ4 ? 5 : kQ8 ? 3 : 0;                 // tiles of codes
  static constexpr int kCodeBytes = kQ4 ? kQ4Bytes : kHeadDim;       // of a vector
  static constexpr int kRawBytes = kTile * kCodeBytes;
  static constexpr int kRingAt = kQTiles * kQBytes;
  static constexpr int kRawAt = kRingAt + kStages * kTileBytes;
  static constexpr int kTileArea = kRawAt + kRaw * kRawBytes;
  static constexpr uint32_t kTmemCols = 256 * kGroups;
  static constexpr int kOAt = 128 * kGroups;  // O's columns
  static constexpr int kSegs = kMode == kWide ? 32 : kQ8 ? 12 : 10;
};

template <int kMode> struct Control {
  using Sh = Shape<kMode>;
  uint64_t full[Sh::kStages], empty[Sh::kStages];
  uint64_t raw_full[Sh::kQ8 ? Sh::kRaw : 1], raw_empty[Sh::kQ8 ? Sh::kRaw : 1];
  uint64_t q_full[2], q_free[2], s_full[2], p_half[2], p_full[2], o_done[2], mend[2], mended[2];
  uint64_t joined, read, drain;
  uint32_t tmem;
  int abort;      // a wait ran out: every role leaves
  int poison;     // a non-finite V was zeroed in some tile
  int pad;
  uint8_t bad[8];  // per tile, bit i: tokens 16 i .. + 15 have no page
  ChunkShare<Sh::kSegs> share;
  union {
    int red[32];                         // share_init
    float2 ml[2][Sh::kTurns ? Sh::kRows : 1];  // maximum and sum of each group's rows
  };
  // per tile of codes: its scale bytes, and its rows that hold a token
  alignas(16) uint8_t scale[Sh::kQ8 ? Sh::kRaw : 1][Sh::kQ8 ? kTile : 16];  // 4-bit: powers
  alignas(16) uint8_t group[Sh::kQ4 ? Sh::kRaw : 1][Sh::kQ4 ? kTile * kQ4Scales : 16];
  int raw_rows[Sh::kQ8 ? Sh::kRaw : 1], raw_bad[Sh::kQ8 ? Sh::kRaw : 1];
};
template <int kMode> constexpr int smem_bytes() {
  return Shape<kMode>::kTileArea + (int)sizeof(Control<kMode>);
}
static_assert(smem_bytes<kWide>() <= 227 * 1024, "shared memory");
static_assert(smem_bytes<kPair>() <= 227 * 1024, "shared memory");
static_assert(smem_bytes<kPair8>() <= 227 * 1024, "shared memory");
static_assert(smem_bytes<kPair4>() <= 227 * 1024, "shared memory");
static_assert(2 * (smem_bytes<kSolo>() + 1024) <= 228 * 1024, "shared memory");

// What the V of a tile needs before the product reads it.
struct Mend {
  int zero_lo, zero_hi;  // token rows past the end in the last page
  // rows that some row of the unit does not see: [0, lo_end) before its last
  // row's window, [hi, hi_end) behind its first row's token
  int lo_end, hi, hi_end;
  __device__ __forceinline__ bool scans() const { return lo_end > 0 || hi < hi_end; }
};
__device__ __forceinline__ Mend mend_of(const ChunkArgs &a, const ChunkSeg &g, int tile) {
  const int tok0 = tile * kTile;
  Mend m{0, 0, 0, 0, 0};
  const int valid = min(kTile, g.len - tok0);
  if (valid <= 0) return m;
  if (valid < kTile && (g.len & (a.ps - 1)) != 0) {
    m.zero_lo = valid;
    m.zero_hi = min(kTile, ((g.len + a.ps - 1) & -a.ps) - tok0);
  }
  m.hi = max(0, g.t_first + 1 - tok0);
  m.hi_end = valid;
  if (a.window > 0) m.lo_end = min(m.hi < valid ? m.hi : valid, g.t_last - a.window + 1 - tok0);
  return m;
}
__device__ __forceinline__ bool at_edge(const ChunkSeg &g, int tile) {
  return tile >= g.edge_from || tile <= g.edge_upto;
}

// the exponent field, and what carries out of it when it is all ones
template <class T> struct NonFinite;
template <> struct NonFinite<__half> {
  static constexpr uint32_t kMask = 0x7C007C00u, kOne = 0x04000400u;
};
template <> struct NonFinite<__nv_bfloat16> {
  static constexpr uint32_t kMask = 0x7F807F80u, kOne = 0x00800080u;
};

__device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t acc, __half) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
  return r;
}
__device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t acc, __nv_bfloat16) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
  return r;
}
// Zeroes the infinities and NaN in rows [r0, r1) of 64 channels of a V tile (the
// warp does it together) and says whether this lane found any.  x * 0 + 0 is
// NaN for those alone, so one packed operation per two elements looks them
// over, with eight sums apart to keep the operations independent.
template <class T>
__device__ __forceinline__ bool clean_rows(uint8_t *slab, int r0, int r1, int lane) {
  bool found = false;
  // where in its row a chunk of 16 bytes sits does not matter here
  uint4 *at = reinterpret_cast<uint4 *>(slab) + r0 * 8;
  const int chunks = (r1 - r0) * 8;
#pragma unroll 1
  for (int i0 = lane; i0 < chunks; i0 += 256) {
    uint32_t acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (i0 + 32 * k < chunks) {
        const uint4 w = at[i0 + 32 * k];
        acc[(2 * k) & 7] = times_zero(w.x, acc[(2 * k) & 7], T{});
        acc[(2 * k + 1) & 7] = times_zero(w.y, acc[(2 * k + 1) & 7], T{});
        acc[(2 * k) & 7] = times_zero(w.z, acc[(2 * k) & 7], T{});
        acc[(2 * k + 1) & 7] = times_zero(w.w, acc[(2 * k + 1) & 7], T{});
      }
    }
    uint32_t any = 0;  // NaN has bits, +-0 at most the signs
#pragma unroll
    for (int k = 0; k < 8; ++k) any |= acc[k] & 0x7FFF7FFFu;
    if (!any) continue;
    found = true;
    constexpr uint32_t M = NonFinite<T>::kMask, O = NonFinite<T>::kOne;
#pragma unroll 1
    for (int i = i0; i < min(chunks, i0 + 256); i += 32) {
      uint32_t *u = reinterpret_cast<uint32_t *>(at + i);
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const uint32_t b = ((u[k] & M) + O) & 0x80008000u;
        if (b & 0x8000u) u[k] &= 0xFFFF0000u;
        if (b & 0x80000000u) u[k] &= 0x0000FFFFu;
      }
    }
  }
  return found;
}

// Writes over channels [c0, c1) of each lane's row, the unit's row r, where it sees
// infinities or NaN of V; 8-bit: NaN, where it sees a NaN vector.  A warp's lanes look the
// cache over together: all tiles of the segment, or those that were scanned, which alone
// can hold such values where every result is finite.  need: the row is there and its
// weights are not NaN.
template <class T, bool kQ8>
__device__ __forceinline__ void put_odd(const ChunkArgs &a, const ChunkSeg &g, int r, int c0, int c1,
                                        bool need, bool all) {
  const int lane = threadIdx.x & 31;
  const int t = g.len - g.n + token_of(a, g.r0 + r), from = a.window > 0 ? t - a.window + 1 : 0;
  Odd row[4];  // of channels 32 i .. + 31
#pragma unroll 1
  for (int tile = g.tile_lo; tile < g.tile_hi; ++tile) {
    if (!kQ8 && !all && !mend_of(a, g, tile).scans()) continue;
#pragma unroll 1
    for (int j0 = tile * kTile; j0 < min(g.len, (tile + 1) * kTile); j0 += 16) {
      const int ph = a.bt[(long long)g.b * a.maxP + j0 / a.ps];
      if (ph < 0 || ph >= a.nphys) continue;
      const long long vec = ((long long)ph * a.Hkv + g.kvh) * a.ps + (j0 & (a.ps - 1));
      if constexpr (kQ8) {
        uint32_t nan = __ballot_sync(0xFFFFFFFFu, a.v_scale[vec + (lane & 15)] == kQ8NanScale);
        for (nan &= 0xFFFFu; nan; nan &= nan - 1) {
          const int j = j0 + __ffs(nan) - 1;
          if (j <= t && j >= from)
#pragma unroll
            for (int i = 0; i < 4; ++i) row[i].plus = row[i].minus = ~0u;
        }
      } else {
        // half a warp reads a vector
        const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.v) +
                                                         vec * kHeadDim) + lane;
        uint4 w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = v[32 * k];
        Odd eight[8];  // of this lane's channels of token 2 k + (lane >> 4)
        uint32_t some = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float x[8];
          load8(reinterpret_cast<const T *>(&w[k]), x);
#pragma unroll
          for (int i = 0; i < 8; ++i) eight[k].see(i, x[i]);
          some |= (eight[k].plus | eight[k].minus) ? 1u << k : 0u;
        }
        some = __reduce_or_sync(0xFFFFFFFFu, some);
        if (!some) continue;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (!((some >> k) & 1)) continue;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const int j = j0 + 2 * k + h;
            const bool sees = j <= t && j >= from;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool mine = lane >> 2 == 4 * h + i;
              const uint32_t plus = __reduce_or_sync(
                  0xFFFFFFFFu, mine ? eight[k].plus << (8 * (lane & 3)) : 0u);
              const uint32_t minus = __reduce_or_sync(
                  0xFFFFFFFFu, mine ? eight[k].minus << (8 * (lane & 3)) : 0u);
              if (sees) row[i].plus |= plus, row[i].minus |= minus;
            }
          }
        }
      }
    }
  }
  if (!need) return;
  T *out = static_cast<T *>(a.out) + row_offset(a, g.q0, g.kvh, g.r0 + r);
  float *part =
      g.whole() ? nullptr : a.part_o + ((long long)part_slot(g) * a.slot_rows + r) * kHeadDim;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll 1
    for (int c = max(c0, 32 * i); c < min(c1, 32 * i + 32); ++c) {
      if (!row[i].any(c & 31)) continue;
      const float x = row[i].sum(c & 31);
      if (part) part[c] = x;
      else out[c] = (T)x;
    }
}

// The same for a list of segments, once all are written: the group's rows start at row
// r_lo of a unit.  Bit i of `odd` and `nan`: in segment i a result of the lane's row is not
// finite, its weights are NaN.  (Where a segment is written, a call costs the registers
// of what goes on there: 32 prompts of 512 80 -> 85 us.)
template <class T, bool kQ8>
__device__ __noinline__ void put_odd_list(const ChunkArgs &a, const ChunkSeg *seg, int nseg, int r_lo,
                                          int c0, int c1, uint32_t odd, uint32_t nan, bool zeroed) {
  const int row = threadIdx.x & 127;
  for (int i = 0; i < nseg; ++i) {
    const bool need = row < a.row_tile && r_lo + row < seg[i].nrows && !((nan >> i) & 1);
    const bool all = __any_sync(0xFFFFFFFFu, need && ((odd >> i) & 1));
    if (!all && !(zeroed && __any_sync(0xFFFFFFFFu, need))) continue;
    put_odd<T, kQ8>(a, seg[i], min(r_lo + row, seg[i].nrows - 1), c0, c1, need, all);
  }
}

// bits lo .. hi of 32 columns, less those of the two 16-token pages in `bad`
__device__ __forceinline__ uint32_t visible_bits(int lo, int hi, uint32_t bad) {
  const uint32_t upto = hi < 0 ? 0u : hi >= 31 ? ~0u : (2u << hi) - 1u;
  const uint32_t from = lo <= 0 ? ~0u : lo > 31 ? 0u : ~0u << lo;
  const uint32_t out = ((bad & 1) ? 0xFFFFu : 0u) | ((bad & 2) ? 0xFFFF0000u : 0u);
  return upto & from & ~out;
}

template <class T> __device__ __forceinline__ constexpr float weight_bias() { return 0.f; }
template <> __device__ __forceinline__ constexpr float weight_bias<__half>() { return 7.f; }

// 16 codes times a power of two, as 16 elements of T.  f16: the hardware's
// conversion and a multiplication.
template <class T> __device__ __forceinline__ uint32_t q8_factor(uint32_t byte);
template <> __device__ __forceinline__ uint32_t q8_factor<__half>(uint32_t byte) {
  const uint32_t h = pack2(q8_scale(byte), 0.f, __half{}) & 0xFFFFu;
  return h | (h << 16);
}
__device__ __forceinline__ void q8_expand(uint4 w, uint32_t f, uint32_t (&x)[8], __half) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a, b;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)(u[i] & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(u[i] >> 16)));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(x[2 * i]) : "r"(a), "r"(f));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(x[2 * i + 1]) : "r"(b), "r"(f));
  }
}
// bf16: a code's exponent and mantissa, moved to where bf16 has them, are the
// code times 2^-120 (subnormal codes too: they become subnormal bf16), so one
// exact multiplication by 2^(e + 120), e + 120 <= 127, gives the value.
template <> __device__ __forceinline__ uint32_t q8_factor<__nv_bfloat16>(uint32_t byte) {
  const uint32_t h = byte == (uint32_t)kQ8NanScale ? 0x7FFFu : min(byte + 120u, 254u) << 7;
  return h | (h << 16);
}
__device__ __forceinline__ void q8_expand(uint4 w, uint32_t f, uint32_t (&x)[8], __nv_bfloat16) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the low and the high byte of each of the four results, then two by two
    const uint32_t lo = (u[i] & 0x0F0F0F0Fu) << 4;
    const uint32_t hi = (u[i] & 0x80808080u) | ((u[i] >> 4) & 0x07070707u);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(x[2 * i]) : "r"(__byte_perm(lo, hi, 0x5140)), "r"(f));
    asm("mul.rn.bf16x2 %0, %1, %2;"
        : "=r"(x[2 * i + 1])
        : "r"(__byte_perm(lo, hi, 0x7362)), "r"(f));
  }
}

// A warp copies the scales and powers of a tile of 4-bit K (w = 0) or V, from the page rows that
// lane i has in y (rows_total: no page).  (As bulk copies, three a page with the codes', they bound
// pages of 16 tokens.)
__device__ __forceinline__ void copy_q4_scales(const ChunkArgs &a, int w, int y, int rows_total,
                                               uint32_t groups, uint32_t powers) {
  const int lane = threadIdx.x & 31, log2 = 31 - __clz(a.ps);
#pragma unroll
  for (int i = 0; i < 3; ++i) {  // the scales of 64 tokens, 64 more, and the powers
    const int token = i < 2 ? 64 * i + 2 * lane : 16 * (lane & 7);
    const int page = __shfl_sync(0xFFFFFFFFu, y, token >> log2);
    const long long row = page + (token & (a.ps - 1));
    if (page == rows_total) continue;
    if (i < 2)
      cp_async16(groups + token * kQ4Scales, (w ? a.v_group : a.k_group) + row * kQ4Scales);
    else if (lane < kTile / 16)
      cp_async16(powers + token, (w ? a.v_scale : a.k_scale) + row);
  }
}

template <class T, int kMode>
__global__ void __launch_bounds__(Shape<kMode>::kThreads, Shape<kMode>::kCtas)
    chunk_mma_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ CUtensorMap tq,
                     const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv) {
  using Sh = Shape<kMode>;
  constexpr bool kHalves = Sh::kHalves, kTurns = Sh::kTurns, kQ8 = Sh::kQ8, kQ4 = Sh::kQ4;
  constexpr int kLoad = 4 * Sh::kGroups;  // the loader's warp; the others' follow
  constexpr int kOAt = Sh::kOAt;
  constexpr int kStages = Sh::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *q_area = smem;
  uint8_t *ring = smem + Sh::kRingAt;
  Control<kMode> &ctl = *reinterpret_cast<Control<kMode> *>(smem + Sh::kTileArea);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it
    if (tid == 0) flag_error(a.status, KV_ERR_INVALID_ARG);
    return;
  }
  if (warp == kLoad + 1) tmem_alloc(smem_u32(&ctl.tmem), Sh::kTmemCols);
  if (tid == 0) {
    if (!kQ8) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tk)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tv)) : "memory");
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&ctl.full[i]), kQ8 ? 4 : 1);
      mbar_init(smem_u32(&ctl.empty[i]), 1);
    }
    for (int i = 0; i < Sh::kRaw; ++i) {
      mbar_init(smem_u32(&ctl.raw_full[i]), kQ4 ? 33 : 1);  // (4 bits: a lane's small copies each)
      mbar_init(smem_u32(&ctl.raw_empty[i]), 4);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&ctl.q_full[x]), 1);
      mbar_init(smem_u32(&ctl.q_free[x]), 1);
      mbar_init(smem_u32(&ctl.s_full[x]), 1);
      mbar_init(smem_u32(&ctl.p_half[x]), 4);
      mbar_init(smem_u32(&ctl.p_full[x]), 4);
      mbar_init(smem_u32(&ctl.o_done[x]), 1);
      mbar_init(smem_u32(&ctl.mend[x]), 1);
      mbar_init(smem_u32(&ctl.mended[x]), 2);
    }
    mbar_init(smem_u32(&ctl.joined), 8);
    mbar_init(smem_u32(&ctl.read), 8);
    mbar_init(smem_u32(&ctl.drain), 1);
    fence_mbar_init();
    ctl.abort = 0;
    ctl.poison = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  pdl_wait();
  if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  const int rt = a.row_tile, unit_rows = rt * Sh::kQTiles;
  share_init(a, unit_rows, kTile, &ctl.share, ctl.red);
  const Waiter wait{&ctl.abort, a.wait_limit_ns};
  const auto &share = ctl.share;
  const int group = Sh::kGroups == 1 ? 0 : warp >> 2;  // softmax group

  // state that lives across lists of segments
  Ring<kStages> ld;              // loader: next slot; menders: the next tile's K slot
  Ring<kQ8 ? Sh::kRaw : 1> raw;  // loader and converter: next tile of codes
  Ring<kStages> qk, pv;          // products: slot of the next K / of the next tile's K
  uint32_t tiles_loaded = 0;     // loader, softmax: tiles so far
  uint32_t q_ph = 0, p_ph = 0, mend_ph = 0;  // bit x
  uint32_t s_ph = 0, o_ph = 0, j_ph = 0;
  uint32_t q_uses = 0;           // bit x: the Q tile has been used before

  // the next list of segments; all threads ask together
  auto next_list = [&](bool list) -> bool {
    __syncthreads();
    if (list && tid == 0) {
      share_next(a, unit_rows, kTile, &ctl.share);
      if (*reinterpret_cast<volatile int *>(&ctl.abort)) ctl.share.nseg = 0;
    }
    __syncthreads();
    return share.nseg != 0;
  };

  // registers: 256 threads x 200 + 128 x 104 = 384 x 168, 256 x 184 + 256 x 72 = 512
  // x 128 and 128 x 184 + 128 x 72 = 256 x 128, the launch's; the four warps of a
  // warpgroup change theirs together
  if (warp < kLoad) {
    if constexpr (kQ8 || kMode == kSolo) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
  } else {
    if constexpr (kQ8 || kMode == kSolo) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
  }
  if (warp < kLoad) {
    // --------------------------------------------------------------- softmax
    while (next_list(true)) {
      const int x = group;
      const int row = (warp & 3) * 32 + lane;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t s_at = tmem + lanes + x * 128, o_at = tmem + lanes + kOAt + x * 128;
      // (the Q loader has seen to the sign of the scale, and to 0)
      const float sc = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);
      bool live = true;
      uint32_t odd_segs = 0, nan_segs = 0;  // for put_odd_list
      static_assert(Sh::kSegs <= 32, "bits");
      const int nseg = share.nseg;
      for (int sg = 0; sg < nseg && live; ++sg) {
        const ChunkSeg g = share.seg[sg];
        const int r_lo = kHalves ? x * rt : 0;  // the group's rows of the unit
        const int urow = r_lo + row;
        const bool mine = row < rt && urow < g.nrows;
        // the first group's rows see no tile from half_hi on
        const int end = kHalves && x == 0 ? min(g.tile_hi, g.half_hi) : g.tile_hi;
        const bool active = !kHalves || (x == 0 ? r_lo < g.nrows : g.nrows > rt);
        if (!active) {
          tiles_loaded += g.tile_hi - g.tile_lo;
          continue;
        }
        const bool any_row = (warp & 3) * 32 < min(rt, g.nrows - r_lo);
        const int t = g.len - g.n + token_of(a, g.r0 + min(urow, g.nrows - 1));
        float m = -INFINITY, l = 0.f;
        bool begun = false;
        for (int tile = g.tile_lo + (kTurns ? x : 0); tile < end; tile += kTurns ? 2 : 1) {
          if (!wait(smem_u32(&ctl.s_full[x]), s_ph)) {
            live = false;
            break;
          }
          s_ph ^= 1;
          // (and every product issued before: O holds the tiles before this one)
          const uint32_t seq = tiles_loaded + (uint32_t)(tile - g.tile_lo);
          if (any_row) {
            tc_fence_after();
            float s[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, s + 32 * c);
            tc_wait_ld();
            const int tok0 = tile * kTile;
            const int hi = vis_hi(t, tok0), lo = vis_lo(t, tok0, a.window);
            const uint32_t bad = ctl.bad[seq & 7];
            if (!__all_sync(0xFFFFFFFFu, hi >= kTile - 1 && lo <= 0) || bad) {
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t see = visible_bits(lo - 32 * w, hi - 32 * w, bad >> (2 * w));
                if (__all_sync(0xFFFFFFFFu, see == ~0u)) continue;
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  s[32 * w + c] = (see >> c) & 1 ? s[32 * w + c] : -INFINITY;
              }
            }
            float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
#pragma unroll
            for (int c = 4; c < 124; c += 8) {
              mx0 = max3(mx0, s[c], s[c + 1]);
              mx1 = max3(mx1, s[c + 2], s[c + 3]);
              mx2 = max3(mx2, s[c + 4], s[c + 5]);
              mx3 = max3(mx3, s[c + 6], s[c + 7]);
            }
            mx0 = max3(mx0, s[124], s[125]);
            mx1 = max3(mx1, s[126], s[127]);
            const float mx = fmaxf(max3(mx0, mx1, mx2), mx3);
            // m = -inf: nothing seen so far (a difference of two -inf is NaN: no move)
            const bool move = (mx - m) * sc > kMoveAt;
            if (begun && __any_sync(0xFFFFFFFFu, move)) {
              const float alpha = !move ? 1.f : m == -INFINITY ? 0.f : ex2((m - mx) * sc);
              l *= alpha;
#pragma unroll 1
              for (int c = 0; c < kHeadDim; c += 32) {
                float o[32];
                tmem_ld32(o_at + c, o);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= alpha;
                tmem_st32(o_at + c, o);
              }
            }
            if (move) m = mx;
            const float base = m == -INFINITY ? 0.f : m * sc - weight_bias<T>();
            const uint64_t sc2 = f2_pack(sc, sc), base2 = f2_pack(-base, -base);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t p[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float &p0 = s[32 * c + 2 * i], &p1 = s[32 * c + 2 * i + 1];
                f2_unpack(f2_fma(f2_pack(p0, p1), sc2, base2), p0, p1);
                p0 = ex2(p0);
                p1 = ex2(p1);
                p[i] = pack2(p0, p1, T{});
              }
              tmem_st16(s_at + 16 * c, p);
              if (c == 1) {
                // the product starts with the first 64 tokens' weights
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl.p_half[x]));
              }
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl.p_full[x]));
            // the sum, while the product runs
            uint64_t sum[4] = {0, 0, 0, 0};  // pairs of zeros
#pragma unroll
            for (int c = 0; c < 128; c += 2)
              sum[(c >> 1) & 3] = f2_add(sum[(c >> 1) & 3], f2_pack(s[c], s[c + 1]));
            float sum0, sum1;
            f2_unpack(f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3])), sum0, sum1);
            l += sum0 + sum1;
          } else if (lane == 0) {
            mbar_arrive(smem_u32(&ctl.p_half[x]));
            mbar_arrive(smem_u32(&ctl.p_full[x]));
          }
          begun = true;
        }
        if (!live) break;
        tiles_loaded += g.tile_hi - g.tile_lo;
        if (begun) {
          if (!wait(smem_u32(&ctl.o_done[x]), o_ph)) {
            live = false;
            break;
          }
          o_ph ^= 1;
        }
        tc_fence_after();
        float M = m == -INFINITY ? -INFINITY : m * sc - weight_bias<T>();
        const bool whole = g.whole();
        const int pr = g.r0 + min(urow, g.nrows - 1);
        T *out = static_cast<T *>(a.out) + row_offset(a, g.q0, g.kvh, pr);
        float *part = nullptr;
        long long prow = 0;
        if (!whole) {
          prow = (long long)part_slot(g) * a.slot_rows + min(urow, g.nrows - 1);
          part = a.part_o + prow * kHeadDim;
        }
        float f0 = 1.f, f1 = 0.f;
        // the row saw nothing, or O is not there (of NaN scores alone, l is NaN)
        bool none0 = m == -INFINITY && l == 0.f, none1 = true;
        constexpr int kCols = kTurns ? 64 : 128;  // channels this thread writes
        const int c0 = kTurns ? 64 * x : 0;
        const bool second = kTurns && g.tile_hi - g.tile_lo > 1;
        if constexpr (kTurns) {
          // both groups hold part of every row: each writes half the channels
          if (any_row) ctl.ml[x][row] = make_float2(M, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl.joined));
          if (!wait(smem_u32(&ctl.joined), j_ph)) {
            live = false;
            break;
          }
          tc_fence_after();
          const int at = any_row ? row : 0;
          const float2 u = ctl.ml[0][at], v = ctl.ml[1][at];
          M = fmaxf(u.x, v.x);
          const float b = M == -INFINITY ? 0.f : M;
          none0 = u.x == -INFINITY && u.y == 0.f;
          none1 = v.x == -INFINITY && v.y == 0.f;
          f0 = ex2(u.x - b);
          f1 = ex2(v.x - b);
          l = u.y * f0 + v.y * f1;
        }
        if (any_row) {
          const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;  // (a part stays as it is)
          f0 *= inv;
          f1 *= inv;
          const uint32_t o0 = tmem + lanes + kOAt + (kTurns ? 0 : x * 128) + c0;
          const bool nothing = __any_sync(0xFFFFFFFFu, none0);
          bool odd = false;  // a result is not finite
          // rows of this lane's quad, for the transposed stores
          T *quad_out[4];
          bool quad_mine[4];
          if (whole) {
            const uint32_t valid = __ballot_sync(0xFFFFFFFFu, mine);
            const unsigned long long at = reinterpret_cast<unsigned long long>(out);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int src = (lane & ~3) + k;
              quad_out[k] = reinterpret_cast<T *>(__shfl_sync(0xFFFFFFFFu, at, src));
              quad_mine[k] = (valid >> src) & 1;
            }
          }
          // (code that runs once per unit is kept short: its instructions are
          // fetched each time)
#pragma unroll 1
          for (int c = 0; c < kCols; c += 32) {
            float o[32];
            tmem_ld32(o0 + c, o);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= f0;
            if (nothing && none0) {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = 0.f;
            }
            if (second) {
              float o1[32];
              tmem_ld32(o0 + 128 + c, o1);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] += none1 ? 0.f : o1[i] * f1;
            }
            if (whole) {
              // A lane holds four 16-byte chunks of its row.  Transposed among
              // the quad's lanes, a store writes 64 bytes in a row instead of 16.
              uint32_t h[4][4];  // [chunk][word]
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  h[k][i] = pack2(o[8 * k + 2 * i], o[8 * k + 2 * i + 1], T{});
              if constexpr (!kQ8) {
                uint32_t z[4] = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                  for (int i = 0; i < 4; ++i) z[i] = times_zero(h[k][i], z[i], T{});
                odd |= ((z[0] | z[1] | z[2] | z[3]) & 0x7FFF7FFFu) != 0;
              }
#pragma unroll
              for (int step = 1; step < 4; step *= 2) {
                const bool up = lane & step;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (k & step) continue;
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const uint32_t give = up ? h[k][i] : h[k + step][i];
                    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, give, step);
                    (up ? h[k][i] : h[k + step][i]) = got;
                  }
                }
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)  // row k of the quad, chunk lane & 3
                if (quad_mine[k])
                  *reinterpret_cast<uint4 *>(quad_out[k] + c0 + c + 8 * (lane & 3)) =
                      make_uint4(h[k][0], h[k][1], h[k][2], h[k][3]);
            } else if (mine) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4 *>(part + c0 + c + i) =
                    make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
          }
          if (mine && !whole && (!kTurns || x == 0)) {
            a.part_ml[2 * prow] = M;
            a.part_ml[2 * prow + 1] = l;
          }
          if (odd) odd_segs |= 1u << sg;
          if (l != l) nan_segs |= 1u << sg;
          tc_fence_before();
        }
        if constexpr (kTurns) {
          // O may be overwritten once both groups have read it
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl.read));
          if (!wait(smem_u32(&ctl.read), j_ph)) {
            live = false;
            break;
          }
          j_ph ^= 1;
        }
      }
      __syncwarp();  // (a row's stores were its quad's)
      const bool zeroed = __any_sync(0xFFFFFFFFu, *reinterpret_cast<volatile int *>(&ctl.poison));
      if (live && (zeroed || __any_sync(0xFFFFFFFFu, odd_segs)))  // (seldom)
        put_odd_list<T, kQ8>(a, share.seg, nseg, kHalves ? x * rt : 0, kTurns ? 64 * x : 0,
                             kTurns ? 64 * x + 64 : 128, odd_segs, nan_segs, zeroed);
    }
  } else if (warp == kLoad) {
    // ---------------------------------------------------------------- loader
    while (next_list(false)) {
      const int npg = kTile / a.ps;
      const int rows_total = (int)(a.nphys * a.Hkv * a.ps);
      const uint32_t full0 = smem_u32(&ctl.full[0]), empty0 = smem_u32(&ctl.empty[0]);
      bool live = true;
      const int nseg = share.nseg;
      for (int sg = 0; sg < nseg && live; ++sg) {
        const ChunkSeg g = share.seg[sg];
        const int from = seen_from(a, g);
        // a tile's pages are read while the tile before it is copied
        const auto page_of = [&](int tile) {
          const int page = tile * npg + lane;
          return lane < npg && tile < g.tile_hi && (long long)page * a.ps < g.len
                     ? a.bt[(long long)g.b * a.maxP + page]
                     : -1;
        };
        int ph_next = page_of(g.tile_lo);
        for (int tile = g.tile_lo; tile < g.tile_hi; ++tile, ++tiles_loaded) {
          int y = rows_total;  // past the end: the copy fills zeros
          uint32_t bad = 0;
          const int ph = ph_next;
          ph_next = page_of(tile + 1);
          if (lane < npg) {
            const int page = tile * npg + lane;
            if ((long long)page * a.ps < g.len) {
              if (ph >= 0 && ph < a.nphys) {
                y = (ph * a.Hkv + g.kvh) * a.ps;
              } else {
                if ((page + 1) * a.ps > from) flag_error(a.status, KV_ERR_BOUNDS);
                bad = ((1u << (a.ps / 16)) - 1u) << (lane * (a.ps / 16));
              }
            }
          }
          bad = __reduce_or_sync(0xFFFFFFFFu, bad);
          if constexpr (kQ8) {
            const bool have = y != rows_total;
            const int bytes = __popc(__ballot_sync(0xFFFFFFFFu, have)) * a.ps;
            for (int w = 0; w < 2; ++w, raw.next()) {
              if (!wait(smem_u32(&ctl.raw_empty[raw.s]), raw.ph ^ 1)) {
                live = false;
                break;
              }
              if ((int)tiles_loaded == a.debug_skip_tile) continue;
              const uint32_t bar = smem_u32(&ctl.raw_full[raw.s]);
              if (lane == 0) {
                if (w == 0) ctl.bad[tiles_loaded & 7] = (uint8_t)bad;
                ctl.raw_rows[raw.s] = min(kTile, g.len - tile * kTile);
                ctl.raw_bad[raw.s] = (int)bad;
                mbar_arrive_expect_tx(bar, bytes * (Sh::kCodeBytes + (kQ4 ? 0 : 1)));
              }
              __syncwarp();
              if (have) {
                bulk_load(smem_u32(smem) + Sh::kRawAt + raw.s * Sh::kRawBytes + lane * a.ps * Sh::kCodeBytes,
                          static_cast<const uint8_t *>(w ? a.v : a.k) + (long long)y * Sh::kCodeBytes,
                          a.ps * Sh::kCodeBytes, bar);
                if constexpr (!kQ4)
                  bulk_load(smem_u32(&ctl.scale[raw.s][lane * a.ps]),
                            (w ? a.v_scale : a.k_scale) + y, a.ps, bar);
              }
              if constexpr (kQ4) {
                copy_q4_scales(a, w, y, rows_total, smem_u32(ctl.group[raw.s]),
                               smem_u32(ctl.scale[raw.s]));
                cp_async_arrive_noinc(bar);
              }
            }
          } else {
          for (int w = 0; w < 2; ++w, ld.next()) {
            if (!wait(empty0 + 8 * ld.s, ld.ph ^ 1)) {
              live = false;
              break;
            }
            if ((int)tiles_loaded == a.debug_skip_tile) continue;
            const uint32_t bar = full0 + 8 * ld.s;
            if (lane == 0) {
              if (w == 0) ctl.bad[tiles_loaded & 7] = (uint8_t)bad;
              mbar_arrive_expect_tx(bar, kTileBytes);
            }
            __syncwarp();
            if (lane < npg) {
              const uint32_t dst = smem_u32(ring) + ld.s * kTileBytes + lane * a.ps * 128;
              const CUtensorMap *map = w ? &tv : &tk;
              tma_load_2d(dst, map, 0, y, bar);
              tma_load_2d(dst + kSlab, map, 64, y, bar);
            }
          }
          }
          if (!live) break;
        }
      }
    }
  } else if (warp == kLoad + 1) {
    // -------------------------------------------------------------- products
    // The whole warp walks the list, so that positions and descriptors are
    // uniform values; one lane issues.
    while (next_list(false)) {
      constexpr uint32_t id_qk = umma_idesc<T>(128, 128, false);
      constexpr uint32_t id_pv = umma_idesc<T>(128, 128, true);
      constexpr uint32_t hi = umma_desc_hi(1024);
      constexpr int kQSlab = Sh::kQRows * 128;
      // a position in the list, with what is needed of its segment in registers
      struct Cur {
        int sg, tile, lo, hi, from, upto;
        int hi0;   // end of the first group's tiles
        bool two;  // the second group has rows
      };
      const int nseg = uniform(share.nseg);
      auto enter = [&](Cur &u) {
        if (u.sg >= nseg) return;
        const ChunkSeg &g = share.seg[u.sg];
        u.tile = u.lo = uniform(g.tile_lo);
        u.hi = uniform(g.tile_hi);
        u.from = uniform(g.edge_from);
        u.upto = uniform(g.edge_upto);
        u.two = kHalves && uniform(g.nrows) > rt;
        u.hi0 = u.two ? min(u.hi, uniform(g.half_hi)) : u.hi;
      };
      Cur c, p;  // of the next scores, and of the weights that follow
      c.sg = 0;
      enter(c);
      p = c;
      auto active = [&](int x, const Cur &u) {
        return kTurns ? u.tile + x < u.hi : x == 0 ? u.tile < u.hi0 : kHalves && u.two;
      };
      auto edge = [&](const Cur &u, int tile) { return tile >= u.from || tile <= u.upto; };
      auto advance = [&](Cur &u, Ring<kStages> &r) {
        const int step = kTurns && active(1, u) ? 2 : 1;
        r.next(2 * step);
        u.tile += step;
        if (u.tile >= u.hi) {
          ++u.sg;
          enter(u);
        }
      };
      const uint32_t ctl0 = smem_u32(&ctl);
      auto at = [&](const uint64_t &bar) {
        return ctl0 + (uint32_t)(reinterpret_cast<const uint8_t *>(&bar) -
                                 reinterpret_cast<const uint8_t *>(&ctl));
      };
      const uint32_t full0 = at(ctl.full[0]), empty0 = at(ctl.empty[0]);
      const uint32_t dq = umma_desc_lo(smem_u32(q_area), 16);
      const uint32_t dk = umma_desc_lo(smem_u32(ring), 16);
      const uint32_t dv = umma_desc_lo(smem_u32(ring), kSlab);
      auto issue_qk = [&](auto xc) -> bool {
        constexpr int x = decltype(xc)::value, qx = kTurns ? 0 : x;
        Ring<kStages> r = qk;
        if (kTurns) r.next(2 * x);
        if (c.tile == c.lo && (!kTurns || x == 0)) {
          if (!wait(at(ctl.q_full[qx]), (q_ph >> qx) & 1)) return false;
          q_ph ^= 1u << qx;
        }
        const int tile = c.tile + (kTurns ? x : 0);
        const bool leads = !kHalves || x == 0 || !active(0, c);  // first to use this K
        if (!kQ8 && leads && edge(c, tile) && elect_one()) mbar_arrive(at(ctl.mend[kTurns ? x : 0]));
        __syncwarp();
        if (leads && !wait(full0 + 8 * r.s, r.ph)) return false;
        tc_fence_after();
        const uint32_t a0 = dq + qx * (Sh::kQBytes >> 4), b0 = dk + r.s * (kTileBytes >> 4);
        const bool last = tile + 1 == (x == 0 && kHalves ? c.hi0 : c.hi);
        const bool frees = !kHalves || x == 1 || !c.two;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma_ss(tmem + x * 128, a0 + (((k >> 2) * kQSlab + (k & 3) * 32) >> 4),
                    b0 + (((k >> 2) * kSlab + (k & 3) * 32) >> 4), hi, hi, id_qk, k > 0);
          // (also says that every product issued before is done)
          tc_commit(at(ctl.s_full[x]));
          if (last) tc_commit(at(ctl.q_free[qx]));
          if (frees) tc_commit(empty0 + 8 * r.s);
        }
        __syncwarp();
        return true;
      };
      auto issue_pv = [&](auto xc) -> bool {
        constexpr int x = decltype(xc)::value;
        Ring<kStages> r = pv;
        r.next(1 + (kTurns ? 2 * x : 0));
        const int tile = p.tile + (kTurns ? x : 0);
        if (!kHalves || x == 0 || !active(0, p)) {  // first to use this V
          constexpr int mx = kTurns ? x : 0;
          if (!wait(full0 + 8 * r.s, r.ph)) return false;
          if (!kQ8 && edge(p, tile)) {
            if (!wait(at(ctl.mended[mx]), (mend_ph >> mx) & 1)) return false;
            mend_ph ^= 1u << mx;
          }
        }
        const uint32_t b0 = dv + r.s * (kTileBytes >> 4);
        const uint32_t add = p.tile > p.lo;
        const bool last = tile + (kTurns ? 2 : 1) >= (x == 0 && kHalves ? p.hi0 : p.hi);
        const bool frees = !kHalves || x == 1 || !p.two;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!wait(h ? at(ctl.p_full[x]) : at(ctl.p_half[x]), (p_ph >> x) & 1)) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 4 * h; k < 4 * h + 4; ++k)
              umma_ts(tmem + kOAt + x * 128, tmem + x * 128 + k * 8, b0 + k * (2048 >> 4), hi,
                      id_pv, k > 0 ? 1u : add);
            if (h) {
              if (last) tc_commit(at(ctl.o_done[x]));
              if (frees) tc_commit(empty0 + 8 * r.s);
            }
          }
          __syncwarp();
        }
        p_ph ^= 1u << x;
        return true;
      };
      // Step by step: the products of tile p's weights, and the scores of the
      // tile behind it.  Those of a new unit come only behind both of p's: they
      // wait for its Q.
      const std::integral_constant<int, 0> x0;
      const std::integral_constant<int, 1> x1;
      bool have = false;
      while (have || c.sg < nseg) {
        const bool more = c.sg < nseg, same = have && more && c.sg == p.sg;
        if (have && active(0, p) && !issue_pv(x0)) break;
        if (same && active(0, c) && !issue_qk(x0)) break;
        if (have && active(1, p) && !issue_pv(x1)) break;
        if (same && active(1, c) && !issue_qk(x1)) break;
        if (more && !same &&
            ((active(0, c) && !issue_qk(x0)) || (active(1, c) && !issue_qk(x1))))
          break;
        p = c;
        pv = qk;
        have = more;
        if (more) advance(c, qk);
      }
    }
  } else if (kQ8 && warp >= kLoad + 4) {
    // ------------------------------------------------------------- converter
    // A thread takes 16 codes of a token at a time, eight times per tile: eight
    // lanes read a row of codes, and write two 16-byte chunks each into the
    // row's two swizzled slabs.
    if constexpr (kQ8) {
      const int ct = tid - 384, c16 = ct & 7, row0 = ct >> 3;
      [[maybe_unused]] const Q4Bits<T> bits;
      while (next_list(false)) {
        bool live = true;
        const int nseg = share.nseg;
        for (int sg = 0; sg < nseg && live; ++sg) {
          const int tiles = share.seg[sg].tile_hi - share.seg[sg].tile_lo;
          for (int i = 0; i < 2 * tiles; ++i, ld.next(), raw.next()) {
            if (!wait(smem_u32(&ctl.raw_full[raw.s]), raw.ph) ||
                !wait(smem_u32(&ctl.empty[ld.s]), ld.ph ^ 1)) {
              live = false;
              break;
            }
            // rows row0 + 16 j: they share their swizzle
            const uint8_t *scale = ctl.scale[raw.s] + row0;
            uint8_t *slab = ring + ld.s * kTileBytes + (c16 >> 2) * kSlab;
            uint8_t *to0 = slab + swz(row0, (c16 & 3) * 2), *to1 = slab + swz(row0, (c16 & 3) * 2 + 1);
            bool nan = false;
            // four rows' codes are read ahead of their use (4 x 32k tokens, 32 rows,
            // bf16, 85 -> 74 us; the order that spares the stores' two-way bank
            // conflicts costs more in selections: 74 against 69)
            using Codes = std::conditional_t<kQ4, uint2, uint4>;
            const Codes *codes = reinterpret_cast<const Codes *>(smem + Sh::kRawAt +
                                                                 raw.s * Sh::kRawBytes) + ct;
            Codes codes_of[4];
            uint32_t scale_of[4], group_of[4];
            const uint8_t *group = ctl.group[kQ4 ? raw.s : 0] + row0 * kQ4Scales + c16;
            auto fetch = [&](int r) {
              codes_of[r & 3] = codes[r * 128];
              scale_of[r & 3] = scale[16 * r];
              if constexpr (kQ4) group_of[r & 3] = group[16 * r * kQ4Scales];
            };
#pragma unroll
            for (int r = 0; r < 4; ++r) fetch(r);
#pragma unroll
            for (int r = 0; r < kTile / 16; ++r) {
              const Codes w = codes_of[r & 3];
              const uint32_t byte = scale_of[r & 3], factor = group_of[r & 3];
              if (r + 4 < kTile / 16) fetch(r + 4);
              uint32_t x[8];
              if constexpr (kQ4) {
                const float f = e4m3_pair(factor).x * q4_power(byte);
                const uint32_t ff = pack2(f, f, T{});
                const uint4 lo = bits.expand(w.x, ff), hi = bits.expand(w.y, ff);
                x[0] = lo.x; x[1] = lo.y; x[2] = lo.z; x[3] = lo.w;
                x[4] = hi.x; x[5] = hi.y; x[6] = hi.z; x[7] = hi.w;
              } else {
                q8_expand(w, q8_factor<T>(byte), x, T{});
              }
              nan |= byte == (uint32_t)kQ8NanScale;
              *reinterpret_cast<uint4 *>(to0 + r * 2048) = make_uint4(x[0], x[1], x[2], x[3]);
              *reinterpret_cast<uint4 *>(to1 + r * 2048) = make_uint4(x[4], x[5], x[6], x[7]);
            }
            // of V, rows without a token and NaN vectors must not meet a weight of 0
            const int rows = ctl.raw_rows[raw.s], bad = ctl.raw_bad[raw.s];
            if ((i & 1) && (nan || rows < kTile || bad != 0)) {
#pragma unroll 1
              for (int r = 0; r < kTile / 16; ++r) {
                const bool token = row0 + 16 * r < rows && !((bad >> r) & 1);
                const bool nan_row = scale[16 * r] == kQ8NanScale;
                if (token && nan_row) *reinterpret_cast<volatile int *>(&ctl.poison) = 1;
                if (token && !nan_row) continue;
                *reinterpret_cast<uint4 *>(to0 + r * 2048) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(to1 + r * 2048) = make_uint4(0, 0, 0, 0);
              }
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(smem_u32(&ctl.full[ld.s]));
              mbar_arrive(smem_u32(&ctl.raw_empty[raw.s]));
            }
          }
        }
      }
    }
  } else {
    // --------------------------------------------------- Q loader and menders
    // Warp 11 loads the segment's Q; then both warps see to V at the edges,
    // 64 channels each.  (A segment's Q waits for the scores of the one before, and
    // those never for more than that segment's own edges.)
    while (next_list(false)) {
      bool live = true;
      const int nseg = share.nseg;
      const int ch = lane & 15, half = lane >> 4;  // 16 bytes of row 2 i + half
      for (int sg = 0; sg < nseg && live; ++sg) {
        const ChunkSeg g = share.seg[sg];
        for (int x = 0; warp == kLoad + 3 && x < Sh::kQTiles && x * rt < g.nrows; ++x) {
          // (the first of two groups may have no tile in this segment)
          if (kHalves && x == 0 && g.nrows > rt && g.tile_lo >= g.half_hi) continue;
          if ((q_uses >> x) & 1) {
            if (!wait(smem_u32(&ctl.q_free[x]), (q_ph >> x) & 1)) {
              live = false;
              break;
            }
            q_ph ^= 1u << x;
          }
          q_uses |= 1u << x;
          if (a.q_tma) {
            // row_tile / G tokens of G heads; behind the sequence's end come
            // rows that nobody reads
            if (lane == 0) {
              const uint32_t bar = smem_u32(&ctl.q_full[x]);
              const uint32_t dst = smem_u32(q_area) + x * Sh::kQBytes;
              const int tok = g.q0 + token_of(a, g.r0 + x * rt);
              mbar_arrive_expect_tx(bar, 2 * rt * 128);
              tma_load_3d(dst, &tq, 0, g.kvh * a.G, tok, bar);
              tma_load_3d(dst + Sh::kQRows * 128, &tq, 64, g.kvh * a.G, tok, bar);
            }
            __syncwarp();
            continue;
          }
          const uint32_t q = smem_u32(q_area) + x * Sh::kQBytes + (ch >> 3) * Sh::kQRows * 128;
          const int pr = g.r0 + x * rt + half, left = min(rt, g.nrows - x * rt);
          int hd = pr - token_of(a, pr) * a.G;
          const T *src = static_cast<const T *>(a.q) + row_offset(a, g.q0, g.kvh, pr) + ch * 8;
          const long long wrap = (long long)(a.Hq - a.G) * kHeadDim;  // to the next token's heads
          for (int r = half; r < Sh::kQRows; r += 2) {
            const uint32_t dst = q + swz(r, ch & 7);
            if (r < left && a.scale_log2 > 0.f) {
              cp_async16(dst, src);
            } else {  // a negative scale turns q, a zero one clears it
              uint4 w = make_uint4(0, 0, 0, 0);
              if (r < left && a.scale_log2 < 0.f) {
                w = *reinterpret_cast<const uint4 *>(src);
                w = make_uint4(w.x ^ 0x80008000u, w.y ^ 0x80008000u, w.z ^ 0x80008000u,
                               w.w ^ 0x80008000u);
              }
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w.x),
                           "r"(w.y), "r"(w.z), "r"(w.w)
                           : "memory");
            }
            src += 2 * kHeadDim;
            hd += 2;
            while (hd >= a.G) {
              hd -= a.G;
              src += wrap;
            }
          }
          cp_async_wait_all();
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl.q_full[x]));
        }
        for (int tile = g.tile_lo; !kQ8 && live && tile < g.tile_hi; ++tile, ld.next(2)) {
          if (!at_edge(g, tile)) continue;
          const Mend m = mend_of(a, g, tile);
          Ring<kStages> r = ld;
          r.next();
          // the product warp asks when it comes to the tile's scores: then the
          // copy of this V is the slot's current or next one
          const int x = kTurns ? (tile - g.tile_lo) & 1 : 0;
          if (!wait(smem_u32(&ctl.mend[x]), (mend_ph >> x) & 1) ||
              !wait(smem_u32(&ctl.full[r.s]), r.ph)) {
            live = false;
            break;
          }
          mend_ph ^= 1u << x;
          uint8_t *v = ring + r.s * kTileBytes + (warp - kLoad - 2) * kSlab;
          for (int i = lane; i < (m.zero_hi - m.zero_lo) * 8; i += 32)
            reinterpret_cast<uint4 *>(v)[m.zero_lo * 8 + i] = make_uint4(0, 0, 0, 0);
          if (m.scans()) {
            bool bad = false;
#pragma unroll 1
            for (int k = 0; k < 2; ++k)
              bad |= clean_rows<T>(v, k ? 0 : m.hi, k ? m.lo_end : m.hi_end, lane);
            if (bad) *reinterpret_cast<volatile int *>(&ctl.poison) = 1;
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl.mended[x]));
        }
      }
    }
  }
  if (ctl.abort) {
    if (tid == 0) flag_error(a.status, KV_ERR_DEVICE_TIMEOUT);
    // leave no copy and no product in flight: every slot's last copy (slots
    // before ld.s were filled in this lap of the ring, the others in the one
    // before), and a last commit
    if (warp == kLoad && kQ8) {
      for (int i = 0; i < Sh::kRaw; ++i)
        mbar_wait(smem_u32(&ctl.raw_full[i]), i < raw.s ? raw.ph : raw.ph ^ 1, drain_limit(a));
    }
    if (warp == kLoad && !kQ8) {
      for (int i = 0; i < kStages; ++i)
        mbar_wait(smem_u32(&ctl.full[i]), i < ld.s ? ld.ph : ld.ph ^ 1, drain_limit(a));
    }
    if (warp == kLoad + 3 && a.q_tma) {
      // q_full's phase in flight: as many as there were uses
      for (int x = 0; x < Sh::kQTiles; ++x)
        if ((q_uses >> x) & 1)
          mbar_wait(smem_u32(&ctl.q_full[x]), (q_ph >> x) & 1, drain_limit(a));
    }
    if (warp == kLoad + 1) {
      if (elect_one()) tc_commit(smem_u32(&ctl.drain));
      mbar_wait(smem_u32(&ctl.drain), 0, drain_limit(a));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kLoad + 1) {
    tc_fence_after();
    tmem_free(tmem, Sh::kTmemCols);
  }
}

template <class T, int kMode>
cudaError_t mma_go(const ChunkArgs &a, const CUtensorMap &tq, const CUtensorMap &tk,
                   const CUtensorMap &tv, int ctas, cudaStream_t st) {
  constexpr int bytes = smem_bytes<kMode>();
  const cudaError_t e = cudaFuncSetAttribute(
      chunk_mma_kernel<T, kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_mma_kernel<T, kMode>, dim3(ctas), dim3(Shape<kMode>::kThreads), bytes,
                    st, a, tq, tk, tv);
}
template <class T>
cudaError_t mma_type(ChunkForm form, const ChunkArgs &a, const CUtensorMap &tq,
                     const CUtensorMap &tk, const CUtensorMap &tv, int ctas, cudaStream_t st) {
  switch (form) {
    case kPair: return mma_go<T, kPair>(a, tq, tk, tv, ctas, st);
    case kPair8: return mma_go<T, kPair8>(a, tq, tk, tv, ctas, st);
    case kPair4: return mma_go<T, kPair4>(a, tq, tk, tv, ctas, st);
    case kSolo: return mma_go<T, kSolo>(a, tq, tk, tv, ctas, st);
    default: return mma_go<T, kWide>(a, tq, tk, tv, ctas, st);
  }
}

}  // namespace

cudaError_t launch_chunk_mma(int dtype, ChunkForm form, const ChunkArgs &a, const CUtensorMap &tq,
                             const CUtensorMap &tk, const CUtensorMap &tv, int ctas,
                             cudaStream_t st) {
  return dtype == KV_F16 ? mma_type<__half>(form, a, tq, tk, tv, ctas, st)
                         : mma_type<__nv_bfloat16>(form, a, tq, tk, tv, ctas, st);
}

}  // namespace kvs
