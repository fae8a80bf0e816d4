// kv_chunk_few.cu -- chunk attention for few rows per kv head (a decode step, a
// few proposed tokens): the 8-bit cache, and 16-bit ones.  kv_chunk.cuh has the
// formula and how the work is cut.
//
// The K/V stream is the bound.  For the 8-bit cache, 33 KB per 128 tokens of K
// and V pass each SM in about 0.75 us at the memory's rate.  Expanding the codes
// into 16-bit tiles in shared memory for the tensor cores' large products
// moves each byte through shared memory seven times and took 2.7 times as long;
// here a warp expands codes in registers, straight into the operands of 16 x 8
// x 16 products, so a byte is written to and read from shared memory once.  For
// 16-bit caches the large products need no expansion and stream as fast over
// long contexts, but their chain of product, softmax and product takes some 2
// us per 128 tokens whatever the rows: here it is a fraction of that, which
// short contexts and many kv heads show.
//
// Measured on one GB300, replayed from a graph: one token over 8 x 65536 tokens, 64/8
// heads, bf16 q, 8-bit: 135 us, 6.1 TB/s of the 6.68 a copy reaches; over 4 x 32768,
// 8-bit: 43 us, with fp32 q 70 us (one CTA per SM); 4 x 700 tokens, 32/8 heads, f16: 9.6
// us, of which the launches, the lengths and the combine are the most (13.6 us as a
// Python call, which the host bounds).
//
// Units of 8 rows (of 16, each byte served two groups of rows, but the registers
// left room for half the warps: slower from 16 rows on).  CTA: four consumer warps
// and a producer warp, two CTAs per SM (one for fp32).  A stage is a 64-token tile
// of K and V (TMA, 128-byte swizzle) and the scale bytes; a consumer warp takes 16
// tokens of it with a softmax of its own; the warps' results are joined at the
// end of a segment.
//   S^T (16 tokens x 8 rows) = K Q^T: the products sum over the channels, in
//     any order that K and Q share: a thread's 16-byte reads of its rows of K
//     are its operands.
//   O^T (128 channels x 8 rows) += V^T P^T: likewise which channel is which row of
//     O^T is free, so a thread reads 16 bytes (twice for 16-bit data) of four
//     tokens and pairs the tokens' elements.
// All swizzled reads meet distinct banks.  For codes the products are f16,
// which holds e4m3 exactly: the scales stay outside.  K's multiplies the scores;
// V's joins the weight's exponent, weight = 2^(z + e_v - R) with R the row's
// running maximum of z + e_v, next to m, that of z, for the softmax's sum: z,
// e_v and both maxima in the log2 domain.  bf16 rows of q are scaled into f16 by a
// power of two per row, which puts the row's largest channel at 2^14: exact for channels
// down to 2^31 below it, with fewer and fewer bits for smaller ones, none from 2^39 on.
// (The power is 2^100 at most: rows below 2^-86 keep fewer bits, of scores below 2^-62
// times the scale.)  fp32 rows of q, and their weights, are taken as two f16 terms (22
// bits), with the value products of each tile summed apart and added in fp32.  The
// other weights enter the value products in 16 bits, f16 over codes and the cache's type
// over 16-bit ones, which is what these products take; a second term would double them.
#include <type_traits>

#include "kv_chunk.cuh"
#include "kv_launch.h"
#include "kv_q8.cuh"
#include "kv_umma.cuh"

namespace kvs {
namespace {

constexpr float kMoveAt = 8.f;  // the maxima move when a weight would exceed 2^8 ...
constexpr float kBias = 7.f;    // ... times 2^7 for f16, so that small weights keep their bits

constexpr int kRows = 8;  // rows of a unit

template <class T, bool Q8> struct Shape {
  static constexpr int kConsumers = 4;
  static constexpr int kThreads = 32 * (kConsumers + 1);
  static constexpr int kTile = 16 * kConsumers;  // tokens per stage
  static constexpr int kRowBytes = kHeadDim * (Q8 ? 1 : 2);
  static constexpr int kSlabs = kRowBytes / 128;
  static constexpr int kBytes = kTile * kRowBytes;  // of K or V
  static constexpr int kStages = Q8 ? 5 : 3;
  static constexpr int kCtas = sizeof(T) == 2 ? 2 : 1;  // per SM
};

template <class T, bool Q8> struct Shared {
  using Sh = Shape<T, Q8>;
  alignas(1024) uint8_t kv[Sh::kStages][2][Sh::kBytes];  // slabs of [token][128 bytes]
  float o[Sh::kConsumers][kRows][kHeadDim];          // per warp, at the end of a segment
  float m[Sh::kConsumers][kRows], r[Sh::kConsumers][kRows], l[Sh::kConsumers][kRows];
  alignas(16) uint8_t scale[Sh::kStages][2][Q8 ? Sh::kTile : 16];
  uint64_t full[Sh::kStages], empty[Sh::kStages], joined, read;
  int tokens[Sh::kStages];  // per stage: bit i: the pages of tokens 16 i .. + 15 are in range
  int abort, pad;
  ChunkShare<Q8 ? 8 : 4> share;
  int red[32];
};

__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, __nv_bfloat16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// which of two packed 16-bit elements are infinities or NaN (bits 15 and 31)
__device__ __forceinline__ uint32_t non_finite(uint32_t w, __half) {
  return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
}
__device__ __forceinline__ uint32_t non_finite(uint32_t w, __nv_bfloat16) {
  return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
// codes 0, 1 (codes 2, 3) of a word as two f16
__device__ __forceinline__ uint32_t f16_lo(uint32_t w) {
  uint32_t x;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x) : "h"((uint16_t)(w & 0xFFFFu)));
  return x;
}
__device__ __forceinline__ uint32_t f16_hi(uint32_t w) {
  uint32_t x;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x) : "h"((uint16_t)(w >> 16)));
  return x;
}

template <class T, bool Q8>
__global__ void __launch_bounds__(Shape<T, Q8>::kThreads, Shape<T, Q8>::kCtas)
    chunk_few_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv) {
  using Sh = Shape<T, Q8>;
  constexpr int kConsumers = Sh::kConsumers, kTile = Sh::kTile, kStages = Sh::kStages;
  constexpr int kSlab = kTile * 128;
  using M = typename std::conditional<Q8, __half, T>::type;  // what the products take
  constexpr bool kTwo = sizeof(T) == 4;                      // q and the weights in two terms
  constexpr int kTerms = kTwo ? 2 : 1;
  constexpr float kShift = std::is_same<M, __half>::value ? kBias : 0.f;
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared<T, Q8> &sh = *reinterpret_cast<Shared<T, Q8> *>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it
    if (tid == 0) flag_error(a.status, KV_ERR_INVALID_ARG);
    return;
  }
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tk)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tv)) : "memory");
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), kConsumers);
    }
    mbar_init(smem_u32(&sh.joined), kConsumers);
    mbar_init(smem_u32(&sh.read), kConsumers);
    fence_mbar_init();
    sh.abort = 0;
  }
  pdl_wait();
  if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  share_init(a, kRows, kTile, &sh.share, sh.red);
  const Waiter wait{&sh.abort, a.wait_limit_ns};
  // the next list of segments; all threads ask together
  auto next_list = [&](bool list) -> bool {
    __syncthreads();
    if (list && tid == 0) {
      share_next(a, kRows, kTile, &sh.share);
      if (*reinterpret_cast<volatile int *>(&sh.abort)) sh.share.nseg = 0;
    }
    __syncthreads();
    return sh.share.nseg != 0;
  };
  Ring<kStages> ring;

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    const int pt = min(a.ps, kTile);  // tokens of a page in a tile
    const int npg = kTile / pt;
    const int rows_total = (int)(a.nphys * a.Hkv * a.ps);
    int filled = 0;
    while (next_list(false)) {
      bool live = true;
      const int nseg = sh.share.nseg;
      for (int sg = 0; sg < nseg && live; ++sg) {
        const ChunkSeg g = sh.share.seg[sg];
        const int from = seen_from(a, g);
        for (int tile = g.tile_lo; tile < g.tile_hi; ++tile, ++filled, ring.next()) {
          int y = rows_total;  // past the end: the copy fills zeros
          uint32_t ok = 0;
          if (lane < npg) {
            const int tok = tile * kTile + lane * pt;
            if (tok < g.len) {
              const int ph = a.bt[(long long)g.b * a.maxP + tok / a.ps];
              if (ph >= 0 && ph < a.nphys) {
                y = (ph * a.Hkv + g.kvh) * a.ps + (tok & (a.ps - 1));
                ok = ((1u << (pt / 16)) - 1u) << (lane * (pt / 16));
              } else if (tok + pt > from) {
                flag_error(a.status, KV_ERR_BOUNDS);
              }
            }
          }
          const int have = __popc(__ballot_sync(0xFFFFFFFFu, ok != 0));
          const uint32_t all = __reduce_or_sync(0xFFFFFFFFu, ok);
          if (!wait(smem_u32(&sh.empty[ring.s]), ring.ph ^ 1)) {
            live = false;
            break;
          }
          if (filled == a.debug_skip_tile) continue;
          const uint32_t bar = smem_u32(&sh.full[ring.s]);
          if (lane == 0) {
            sh.tokens[ring.s] = (int)all;
            mbar_arrive_expect_tx(bar, 2 * Sh::kBytes + (Q8 ? 2 * have * pt : 0));
          }
          __syncwarp();
          if (lane < npg) {
            for (int w = 0; w < 2; ++w) {
              const uint32_t dst = smem_u32(&sh.kv[ring.s][w][lane * pt * 128]);
#pragma unroll
              for (int slab = 0; slab < Sh::kSlabs; ++slab)
                tma_load_2d(dst + slab * kSlab, w ? &tv : &tk, 64 * slab, y, bar);
              if (Q8 && ok)
                bulk_load(smem_u32(&sh.scale[ring.s][w][lane * pt]), (w ? a.v_scale : a.k_scale) + y,
                          pt, bar);
            }
          }
        }
      }
    }
    if (*reinterpret_cast<volatile int *>(&sh.abort)) {
      // leave no copy in flight: each stage's last one (stages before ring.s
      // were filled in this lap, the others in the one before)
      for (int i = 0; i < kStages; ++i)
        mbar_wait(smem_u32(&sh.full[i]), i < ring.s ? ring.ph : ring.ph ^ 1, drain_limit(a));
    }
  } else {
    // ----------------------------------------------------------- consumers
    const int g8 = lane >> 2, t4 = lane & 3;  // row and column group of the fragments
    uint32_t join_ph = 0;
    while (next_list(true)) {
      bool live = true;
      const int nseg = sh.share.nseg;
      for (int sg = 0; sg < nseg && live; ++sg) {
        const ChunkSeg g = sh.share.seg[sg];
        // Q: row n = g8, the 32 channels this thread reads of K's rows,
        // as pairs: codes, 32 t4 .. + 31; 16-bit data, 8 of each of the 16-byte
        // chunks 2 t4, 2 t4 + 1 of both slabs
        uint32_t q[kTerms][16];
        float qf[2];  // scale * log2(e) / the row's power of two, rows 2 t4 and + 1
        int tq[2];    // their tokens
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = 0.f;
        if (g8 < g.nrows) {
          const T *src = static_cast<const T *>(a.q) + row_offset(a, g.q0, g.kvh, g.r0 + g8);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float y[8];
            load8(src + (Q8 ? 32 * t4 + 8 * i : 64 * (i >> 1) + 8 * (2 * t4 + (i & 1))), y);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[8 * i + k] = y[k];
          }
        }
        float f = a.scale_log2;
        if constexpr (Q8 && !std::is_same<T, __half>::value) {
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const int up = top == 0 ? 0 : min(14 - ((int)(top >> 23) - 127), 100);
          const float s = pow2f(up);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] *= s;
          f *= pow2f(-up);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          q[0][i] = pack2(x[2 * i], x[2 * i + 1], M{});
          if constexpr (kTwo) {
            const float2 h = unpack2(q[0][i], M{});
            q[1][i] = pack2(x[2 * i] - h.x, x[2 * i + 1] - h.y, M{});
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          qf[h] = __shfl_sync(0xFFFFFFFFu, f, 4 * (2 * t4 + h));
          tq[h] = g.len - g.n + token_of(a, g.r0 + min(2 * t4 + h, g.nrows - 1));
        }
        float m[2], r[2], l[2], o[8][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          m[h] = r[h] = -INFINITY;
          l[h] = 0.f;
        }
#pragma unroll
        for (int d = 0; d < 8; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[d][i] = 0.f;
        for (int tile = g.tile_lo; tile < g.tile_hi; ++tile, ring.next()) {
          if (!wait(smem_u32(&sh.full[ring.s]), ring.ph)) {
            live = false;
            break;
          }
          const int tok0 = tile * kTile + warp * 16;
          const uint8_t *kc = sh.kv[ring.s][0] + warp * 16 * 128;
          const uint8_t *vc = sh.kv[ring.s][1] + warp * 16 * 128;
          const bool pages = (sh.tokens[ring.s] >> warp) & 1;
          // S^T: tokens g8 and g8 + 8
          float s[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] = 0.f;
#pragma unroll
          for (int c = 0; c < (Q8 ? 2 : 4); ++c) {
            const int at = (c >> 1) * kSlab + g8 * 128 + (((2 * t4 + (c & 1)) ^ g8) << 4);
            const uint4 u = *reinterpret_cast<const uint4 *>(kc + at);
            const uint4 v = *reinterpret_cast<const uint4 *>(kc + at + 8 * 128);
            const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
            // a word of codes is four channels, one step; two words of 16-bit
            // data are
#pragma unroll
            for (int i = 0; i < (Q8 ? 4 : 2); ++i) {
              uint32_t a0, a1, a2, a3;
              if constexpr (Q8) {
                a0 = f16_lo(uu[i]), a2 = f16_hi(uu[i]), a1 = f16_lo(vv[i]), a3 = f16_hi(vv[i]);
              } else {
                a0 = uu[2 * i], a2 = uu[2 * i + 1], a1 = vv[2 * i], a3 = vv[2 * i + 1];
              }
              const int k = Q8 ? 8 * c + 2 * i : 4 * c + 2 * i;
#pragma unroll
              for (int e = kTerms - 1; e >= 0; --e)  // the small term first
                mma16816(s, a0, a1, a2, a3, q[e][k], q[e][k + 1], M{});
            }
          }
          // tokens this thread's lane speaks for: g8 + 8 i
          bool token[2], vbad[2];
          float kf[2], ev[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            token[i] = pages && tok0 + g8 + 8 * i < g.len;
            vbad[i] = !token[i];
            kf[i] = 1.f;
            ev[i] = 0.f;
            if constexpr (Q8) {
              const uint32_t kb = sh.scale[ring.s][0][warp * 16 + g8 + 8 * i];
              const uint32_t vb = sh.scale[ring.s][1][warp * 16 + g8 + 8 * i];
              vbad[i] |= vb == (uint32_t)kQ8NanScale;
              kf[i] = q8_scale(kb);
              ev[i] = vb == (uint32_t)kQ8NanScale ? __uint_as_float(0x7FC00000u)
                                                  : (float)((int)vb - 127);
            }
          }
          const uint32_t bad0 = __ballot_sync(0xFFFFFFFFu, vbad[0]);
          const uint32_t bad1 = __ballot_sync(0xFFFFFFFFu, vbad[1]);
          uint32_t p[kTerms][2];
          float z[4], y[4];  // element i: token g8 + 8 (i >> 1), row 2 t4 + (i & 1)
          bool move = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = i >> 1, h = i & 1;
            const int pos = tok0 + g8 + 8 * k;
            const bool see = token[k] && pos <= tq[h] &&
                             (a.window <= 0 || pos - tq[h] > -a.window);
            z[i] = see ? s[i] * (kf[k] * qf[h]) : -INFINITY;
            y[i] = Q8 && see ? z[i] + ev[k] : z[i];
            move |= z[i] > m[h] + kMoveAt || (Q8 && y[i] > r[h] + kMoveAt);
          }
          if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float mz = fmaxf(z[h], z[h + 2]), my = fmaxf(y[h], y[h + 2]);
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) {
                mz = fmaxf(mz, __shfl_xor_sync(0xFFFFFFFFu, mz, off));
                if (Q8) my = fmaxf(my, __shfl_xor_sync(0xFFFFFFFFu, my, off));
              }
              mz = fmaxf(mz, m[h]);
              my = Q8 ? fmaxf(my, r[h]) : mz;
              // (from -inf: 0, and 1 where it stays there)
              const float al = mz == -INFINITY ? 1.f : ex2(m[h] - mz);
              const float ao = my == -INFINITY ? 1.f : ex2(r[h] - my);
              m[h] = mz;
              r[h] = my;
              l[h] *= al;
#pragma unroll
              for (int d = 0; d < 8; ++d) {
                o[d][h] *= ao;
                o[d][h + 2] *= ao;
              }
            }
          }
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int h = i & 1;
            const float bm = m[h] == -INFINITY ? 0.f : m[h];
            const float br = r[h] == -INFINITY ? 0.f : r[h] - kShift;
            l[h] += ex2(z[i] - bm);
            w[i] = ex2(y[i] - br);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t hi = pack2(w[2 * k], w[2 * k + 1], M{});
            p[0][k] = movm_t(hi);
            if constexpr (kTwo) {
              const float2 h = unpack2(hi, M{});
              p[1][k] = movm_t(pack2(w[2 * k] - h.x, w[2 * k + 1] - h.y, M{}));
            }
          }
          // O^T: tokens 2 t4, 2 t4 + 1 (+ 8); channels 16 g8 .. + 15 of codes, 8 g8
          // .. + 7 of both slabs of 16-bit data
          uint4 v4[Sh::kSlabs][4];
#pragma unroll
          for (int c = 0; c < Sh::kSlabs; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = 2 * t4 + (i & 1) + 8 * (i >> 1);
              v4[c][i] = *reinterpret_cast<const uint4 *>(vc + c * kSlab + row * 128 +
                                                          ((g8 ^ (row & 7)) << 4));
              // rows without a token and NaN vectors must not meet a weight of
              // 0 (a row that sees a NaN vector of codes has a NaN weight);
              // lanes 4 (row & 7) .. speak for the row
              if ((bad0 | bad1) && (((i >> 1 ? bad1 : bad0) >> (4 * (row & 7))) & 1))
                v4[c][i] = make_uint4(0, 0, 0, 0);
            }
          if constexpr (!Q8) {
            // where some row does not see some token, the same holds for
            // infinities and NaN: they are cleared, and the rows that do see
            // them become NaN in their channels, which has the cache read again
            // when they are written (seldom)
            if (tok0 + 15 > g.t_first || a.window > 0) {
              uint32_t any = 0;
#pragma unroll
              for (int c = 0; c < Sh::kSlabs; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  any |= non_finite(v4[c][i].x, M{}) | non_finite(v4[c][i].y, M{}) |
                         non_finite(v4[c][i].z, M{}) | non_finite(v4[c][i].w, M{});
              if (__any_sync(0xFFFFFFFFu, any != 0)) {
                // bit 8 c + 2 k + e of found[i]: element e of word k
                uint32_t found[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  found[i] = 0;
#pragma unroll
                  for (int c = 0; c < Sh::kSlabs; ++c) {
                    uint32_t w[4] = {v4[c][i].x, v4[c][i].y, v4[c][i].z, v4[c][i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                      const uint32_t b = non_finite(w[k], M{});
                      if (b & 0x8000u) w[k] &= 0xFFFF0000u, found[i] |= 1u << (8 * c + 2 * k);
                      if (b & 0x80000000u) w[k] &= 0xFFFFu, found[i] |= 2u << (8 * c + 2 * k);
                    }
                    v4[c][i] = make_uint4(w[0], w[1], w[2], w[3]);
                  }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll 1
                  for (int src = 0; src < 4; ++src) {
                    const uint32_t f = __shfl_sync(0xFFFFFFFFu, found[i], src, 4);
                    const int pos = tok0 + 2 * src + (i & 1) + 8 * (i >> 1);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                      const bool see = pos <= tq[h] &&
                                       (a.window <= 0 || pos - tq[h] > -a.window);
#pragma unroll
                      for (int d = 0; d < 8; ++d) {
                        const float nan = __uint_as_float(0x7FC00000u);
                        if (see && ((f >> (2 * d)) & 1)) o[d][h] = nan;
                        if (see && ((f >> (2 * d)) & 2)) o[d][h + 2] = nan;
                      }
                    }
                  }
                }
              }
            }
          }
          // block d of O^T: of codes, channels 16 g8 + 2 d and + 1; of 16-bit
          // data, 64 (d >> 2) + 8 g8 + 2 (d & 3) and + 1
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            const uint4 *x = v4[Q8 ? 0 : d >> 2];
            const int k = Q8 ? d >> 1 : d & 3;
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = k == 0 ? x[i].x : k == 1 ? x[i].y : k == 2 ? x[i].z : x[i].w;
            uint32_t a0, a1, a2, a3;
            if constexpr (Q8) {
              const uint32_t ab = __byte_perm(w[0], w[1], d & 1 ? 0x7362 : 0x5140);
              const uint32_t cd = __byte_perm(w[2], w[3], d & 1 ? 0x7362 : 0x5140);
              a0 = f16_lo(ab), a1 = f16_hi(ab), a2 = f16_lo(cd), a3 = f16_hi(cd);
            } else {
              a0 = __byte_perm(w[0], w[1], 0x5410), a1 = __byte_perm(w[0], w[1], 0x7632);
              a2 = __byte_perm(w[2], w[3], 0x5410), a3 = __byte_perm(w[2], w[3], 0x7632);
            }
            if constexpr (kTwo) {
              float t[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816(t, a0, a1, a2, a3, p[1][0], p[1][1], M{});
              mma16816(t, a0, a1, a2, a3, p[0][0], p[0][1], M{});
#pragma unroll
              for (int i = 0; i < 4; ++i) o[d][i] += t[i];
            } else {
              mma16816(o[d], a0, a1, a2, a3, p[0][0], p[0][1], M{});
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.empty[ring.s]));
        }
        if (!live) break;
        // elements 0, 1 of o[d]: its even channel, rows 2 t4 and 2 t4 + 1; 2, 3: the odd one
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float lt = l[h];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) lt += __shfl_xor_sync(0xFFFFFFFFu, lt, off);
          const int n = 2 * t4 + h;
#pragma unroll
          for (int d = 0; d < 8; d += 2)
            *reinterpret_cast<float4 *>(
                &sh.o[warp][n][Q8 ? 16 * g8 + 2 * d : 64 * (d >> 2) + 8 * g8 + 2 * (d & 3)]) =
                make_float4(o[d][h], o[d][h + 2], o[d + 1][h], o[d + 1][h + 2]);
          if (g8 == 0) {
            sh.m[warp][n] = m[h];
            sh.r[warp][n] = r[h] == -INFINITY ? -INFINITY : r[h] - kShift;
            sh.l[warp][n] = lt;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.joined));
        if (!wait(smem_u32(&sh.joined), join_ph)) {
          live = false;
          break;
        }
        const bool whole = g.whole();
        for (int n = tid >> 4; n < min(kRows, g.nrows); n += 2 * kConsumers) {
          const int c = (tid & 15) * 8;
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kConsumers; ++w) top = fmaxf(top, sh.m[w][n]);
          const float base = top == -INFINITY ? 0.f : top;
          // (the factors carry V's scales, 2^-110 and up: without 2^64 those of warps whose
          // maximum is 2^-9 below the row's would be 0)
          constexpr float kUp = Q8 ? 64.f : 0.f, kDown = Q8 ? 0x1p-64f : 1.f;
          float sum = 0.f, x[8] = {};
#pragma unroll
          for (int w = 0; w < kConsumers; ++w) {
            sum += sh.l[w][n] * ex2(sh.m[w][n] - base);
            const float f = ex2(sh.r[w][n] - base + kUp);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] += sh.o[w][n][c + k] * f;
          }
          const int pr = g.r0 + n;
          if (whole) {
            if constexpr (!Q8) {
              bool odd = false;
#pragma unroll
              for (int k = 0; k < 8; ++k) odd |= !finite(x[k]);
              if (odd && sum == sum) {  // (seldom)
                const Seen s = seen_tokens(a, g.len - g.n + token_of(a, pr), g.tile_lo, g.tile_hi,
                                           kTile);
                const Odd seen = odd_values<T, 8>(a, g.b, g.kvh, s.lo, s.hi, c);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  if (seen.any(k)) x[k] = seen.sum(k);
              }
            }
            const float inv = sum == 0.f ? 0.f : kDown / sum;
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] *= inv;
            store8(static_cast<T *>(a.out) + row_offset(a, g.q0, g.kvh, pr) + c, x);
          } else {
            const long long at = (long long)part_slot(g) * a.slot_rows + n;
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] *= kDown;
            store8(a.part_o + at * kHeadDim + c, x);
            if (c == 0) {
              a.part_ml[2 * at] = top;
              a.part_ml[2 * at + 1] = sum;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.read));
        if (!wait(smem_u32(&sh.read), join_ph)) {
          live = false;
          break;
        }
        join_ph ^= 1;
      }
    }
  }
  if (tid == 0 && *reinterpret_cast<volatile int *>(&sh.abort))
    flag_error(a.status, KV_ERR_DEVICE_TIMEOUT);
}

template <class T, bool Q8>
cudaError_t few_go(const ChunkArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, int ctas,
                   cudaStream_t st) {
  using Sh = Shape<T, Q8>;
  constexpr int bytes = (int)sizeof(Shared<T, Q8>);
  static_assert(bytes <= (Sh::kCtas == 2 ? 113 : 227) * 1024, "shared memory");
  const cudaError_t e = cudaFuncSetAttribute(
      chunk_few_kernel<T, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_few_kernel<T, Q8>, dim3(ctas), dim3(Sh::kThreads), bytes, st, a, tk,
                    tv);
}

}  // namespace

FewShape chunk_few_shape(int dtype, bool q8) {
  using Own = Shape<__half, false>;
  using Codes = Shape<__half, true>;
  using Codes32 = Shape<float, true>;
  return !q8                ? FewShape{kRows, Own::kTile, Own::kCtas}
         : dtype == KV_F32 ? FewShape{kRows, Codes32::kTile, Codes32::kCtas}
                           : FewShape{kRows, Codes::kTile, Codes::kCtas};
}

cudaError_t launch_chunk_few(int dtype, bool q8, const ChunkArgs &a, const CUtensorMap &tk,
                             const CUtensorMap &tv, int ctas, cudaStream_t st) {
  if (dtype == KV_F32) return few_go<float, true>(a, tk, tv, ctas, st);
  if (dtype == KV_F16)
    return q8 ? few_go<__half, true>(a, tk, tv, ctas, st)
              : few_go<__half, false>(a, tk, tv, ctas, st);
  return q8 ? few_go<__nv_bfloat16, true>(a, tk, tv, ctas, st)
            : few_go<__nv_bfloat16, false>(a, tk, tv, ctas, st);
}

}  // namespace kvs
