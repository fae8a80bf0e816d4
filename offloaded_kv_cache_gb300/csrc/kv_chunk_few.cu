// kv_chunk_few.cu -- chunk attention over the 8-bit cache for few rows per kv
// head (a decode step, a few proposed tokens).  kv_chunk.cuh has the formula
// and how the work is cut.
//
// The codes are the bound: 33 KB per 128 tokens of K and V pass each SM in
// about 0.75 us at the memory's rate.  Expanding them into 16-bit tiles in shared memory
// for the tensor cores' large products moves each byte through shared memory
// seven times and took 2.7 times as long; here a warp expands codes in
// registers, straight into the operands of 16 x 8 x 16 products, so a byte is
// written to and read from shared memory once.
//
// CTA: four consumer warps and a producer warp, two CTAs per SM.  A stage is a
// 64-token tile of K and V codes (TMA, 128-byte swizzle) and their scale bytes; a
// consumer warp takes 16 tokens of it with a softmax of its own; the warps'
// results are joined at the end of a segment.
//   S^T (16 tokens x 8 rows) = K Q^T: the products sum over the channels, in
//     any order that K and Q share: a thread's 16-byte reads of its rows of K
//     are its operands.
//   O^T (128 channels x 8 rows) += V^T P^T: likewise which channel is which row of
//     O^T is free, so a thread reads 16 consecutive codes of four tokens and
//     pairs the tokens' bytes.
// Both swizzled reads meet distinct banks.  Products are f16, which holds e4m3
// exactly: the scales stay outside.  K's multiplies the scores; V's joins the
// weight's exponent, weight = 2^(z + e_v - R) with R the row's running
// maximum of z + e_v, next to m, that of z, for the softmax's sum: z, e_v and
// both maxima in the log2 domain.  bf16 rows of q are scaled into f16 by a power of
// two per row, which is exact but for channels 2^39 below the row's largest.
#include <type_traits>

#include "kv_chunk.cuh"
#include "kv_launch.h"
#include "kv_q8.cuh"
#include "kv_umma.cuh"

namespace kvs {
namespace {

constexpr int kConsumers = 4;
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kTile = 64;                     // tokens per stage, 16 per consumer warp
constexpr int kCodeBytes = kTile * kHeadDim;  // of K or V
constexpr int kStages = 5;
constexpr float kMoveAt = 8.f;  // the maxima move when a weight would exceed 2^8 ...
constexpr float kBias = 7.f;    // ... times 2^7, so that small f16 weights keep their bits

template <int NB> struct Shared {
  alignas(1024) uint8_t code[kStages][2][kCodeBytes];
  float o[kConsumers][8 * NB][kHeadDim];  // per warp, at the end of a segment
  float m[kConsumers][8 * NB], r[kConsumers][8 * NB], l[kConsumers][8 * NB];
  alignas(16) uint8_t scale[kStages][2][kTile];
  uint64_t full[kStages], empty[kStages], joined, read;
  int tokens[kStages];  // per stage: bit i: the pages of tokens 16 i .. + 15 are in range
  int abort, pad;
  ChunkShare<16> share;
  int red[32];
};

__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// Rows of a unit: 8 NB.
template <class T, int NB>
__global__ void __launch_bounds__(kThreads, NB == 1 ? 2 : 1)
    chunk_few_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv) {
  constexpr int kRows = 8 * NB;
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared<NB> &sh = *reinterpret_cast<Shared<NB> *>(smem);
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
        for (int tile = g.tile_lo; tile < g.tile_hi; ++tile, ++filled, ring.next()) {
          int y = rows_total;  // past the end: the copy fills zeros
          uint32_t ok = 0;
          if (lane < npg) {
            const int tok = tile * kTile + lane * pt;
            if (tok < g.len) {
              const int ph = a.bt[(long long)g.b * a.maxP + tok / a.ps];
              if (ph >= 0 && ph < a.nphys) {
                y = (ph * a.Hkv + g.kvh) * a.ps + tok % a.ps;
                ok = ((1u << (pt / 16)) - 1u) << (lane * (pt / 16));
              } else {
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
            mbar_arrive_expect_tx(bar, 2 * kCodeBytes + 2 * have * pt);
          }
          __syncwarp();
          if (lane < npg) {
            tma_load_2d(smem_u32(&sh.code[ring.s][0][lane * pt * kHeadDim]), &tk, 0, y, bar);
            tma_load_2d(smem_u32(&sh.code[ring.s][1][lane * pt * kHeadDim]), &tv, 0, y, bar);
            if (ok) {
              bulk_load(smem_u32(&sh.scale[ring.s][0][lane * pt]), a.k_scale + y, pt, bar);
              bulk_load(smem_u32(&sh.scale[ring.s][1][lane * pt]), a.v_scale + y, pt, bar);
            }
          }
        }
      }
    }
    if (*reinterpret_cast<volatile int *>(&sh.abort)) {
      // leave no copy in flight: each stage's last one (stages before ring.s
      // were filled in this lap, the others in the one before)
      for (int i = 0; i < kStages; ++i)
        mbar_wait(smem_u32(&sh.full[i]), i < ring.s ? ring.ph : ring.ph ^ 1, a.wait_limit_ns);
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
        // Q: row n = 8 nb + g8, channels 32 t4 .. + 31, as f16 pairs
        uint32_t q[NB][16];
        float qf[NB][2];  // scale * log2(e) / the row's power of two, rows 2 t4 and + 1
        int tq[NB][2];    // their tokens
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int n = 8 * nb + g8;
          float x[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0.f;
          if (n < g.nrows) {
            const int pr = g.r0 + n;
            const T *src = static_cast<const T *>(a.q) +
                           ((long long)(g.q0 + pr / a.G) * a.Hq + g.kvh * a.G + pr % a.G) *
                               kHeadDim + 32 * t4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float y[8];
              load8(src + 8 * i, y);
#pragma unroll
              for (int k = 0; k < 8; ++k) x[8 * i + k] = y[k];
            }
          }
          float f = a.scale_log2;
          if constexpr (!std::is_same_v<T, __half>) {
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
          for (int i = 0; i < 16; ++i) q[nb][i] = pack2(x[2 * i], x[2 * i + 1], __half{});
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            qf[nb][h] = __shfl_sync(0xFFFFFFFFu, f, 4 * (2 * t4 + h));
            tq[nb][h] = g.len - g.n + (g.r0 + min(8 * nb + 2 * t4 + h, g.nrows - 1)) / a.G;
          }
        }
        float m[NB][2], r[NB][2], l[NB][2], o[NB][8][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            m[nb][h] = r[nb][h] = -INFINITY;
            l[nb][h] = 0.f;
          }
#pragma unroll
          for (int d = 0; d < 8; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nb][d][i] = 0.f;
        }
        for (int tile = g.tile_lo; tile < g.tile_hi; ++tile, ring.next()) {
          if (!wait(smem_u32(&sh.full[ring.s]), ring.ph)) {
            live = false;
            break;
          }
          const int tok0 = tile * kTile + warp * 16;
          const uint8_t *kc = sh.code[ring.s][0] + warp * 16 * kHeadDim;
          const uint8_t *vc = sh.code[ring.s][1] + warp * 16 * kHeadDim;
          const bool pages = (sh.tokens[ring.s] >> warp) & 1;
          // S^T: tokens g8 and g8 + 8
          float s[NB][4];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nb][i] = 0.f;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int at = g8 * kHeadDim + (((2 * t4 + c) ^ g8) << 4);
            const uint4 u = *reinterpret_cast<const uint4 *>(kc + at);
            const uint4 v = *reinterpret_cast<const uint4 *>(kc + at + 8 * kHeadDim);
            const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t a0 = f16_lo(uu[i]), a2 = f16_hi(uu[i]);
              const uint32_t a1 = f16_lo(vv[i]), a3 = f16_hi(vv[i]);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16816(s[nb], a0, a1, a2, a3, q[nb][8 * c + 2 * i], q[nb][8 * c + 2 * i + 1]);
            }
          }
          uint32_t kb[2], vb[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            kb[i] = sh.scale[ring.s][0][warp * 16 + g8 + 8 * i];
            vb[i] = sh.scale[ring.s][1][warp * 16 + g8 + 8 * i];
          }
          // tokens this thread's lane speaks for: g8 + 8 i
          bool token[2], vbad[2];
          float kf[2], ev[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            token[i] = pages && tok0 + g8 + 8 * i < g.len;
            vbad[i] = !token[i] || vb[i] == (uint32_t)kQ8NanScale;
            kf[i] = q8_scale(kb[i]);
            ev[i] = vb[i] == (uint32_t)kQ8NanScale ? __uint_as_float(0x7FC00000u)
                                                   : (float)((int)vb[i] - 127);
          }
          const uint32_t bad0 = __ballot_sync(0xFFFFFFFFu, vbad[0]);
          const uint32_t bad1 = __ballot_sync(0xFFFFFFFFu, vbad[1]);
          uint32_t p[NB][2];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float z[4], y[4];  // element i: token g8 + 8 (i >> 1), row 2 t4 + (i & 1)
            bool move = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int k = i >> 1, h = i & 1;
              const int pos = tok0 + g8 + 8 * k;
              const bool see = token[k] && pos <= tq[nb][h] &&
                               (a.window <= 0 || pos - tq[nb][h] > -a.window);
              z[i] = see ? s[nb][i] * (kf[k] * qf[nb][h]) : -INFINITY;
              y[i] = see ? z[i] + ev[k] : -INFINITY;
              move |= z[i] > m[nb][h] + kMoveAt || y[i] > r[nb][h] + kMoveAt;
            }
            if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float mz = fmaxf(z[h], z[h + 2]), my = fmaxf(y[h], y[h + 2]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                  mz = fmaxf(mz, __shfl_xor_sync(0xFFFFFFFFu, mz, off));
                  my = fmaxf(my, __shfl_xor_sync(0xFFFFFFFFu, my, off));
                }
                mz = fmaxf(mz, m[nb][h]);
                my = fmaxf(my, r[nb][h]);
                // (from -inf: 0, and 1 where it stays there)
                const float al = mz == -INFINITY ? 1.f : ex2(m[nb][h] - mz);
                const float ao = my == -INFINITY ? 1.f : ex2(r[nb][h] - my);
                m[nb][h] = mz;
                r[nb][h] = my;
                l[nb][h] *= al;
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                  o[nb][d][h] *= ao;
                  o[nb][d][h + 2] *= ao;
                }
              }
            }
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int h = i & 1;
              const float bm = m[nb][h] == -INFINITY ? 0.f : m[nb][h];
              const float br = r[nb][h] == -INFINITY ? 0.f : r[nb][h] - kBias;
              l[nb][h] += ex2(z[i] - bm);
              w[i] = ex2(y[i] - br);
            }
            p[nb][0] = movm_t(pack2(w[0], w[1], __half{}));
            p[nb][1] = movm_t(pack2(w[2], w[3], __half{}));
          }
          // O^T: tokens 2 t4, 2 t4 + 1 (+ 8), channels 16 g8 .. + 15
          uint4 v4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 2 * t4 + (i & 1) + 8 * (i >> 1);
            v4[i] = *reinterpret_cast<const uint4 *>(vc + row * kHeadDim +
                                                     ((g8 ^ (row & 7)) << 4));
          }
          if (bad0 | bad1) {
            // rows without a token and NaN vectors must not meet a weight of 0
            // (a row that sees a NaN vector has a NaN weight)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = 2 * t4 + (i & 1);  // lanes 4 row .. speak for it
              if (((i >> 1 ? bad1 : bad0) >> (4 * row)) & 1) v4[i] = make_uint4(0, 0, 0, 0);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t wa = i == 0 ? v4[0].x : i == 1 ? v4[0].y : i == 2 ? v4[0].z : v4[0].w;
            const uint32_t wb = i == 0 ? v4[1].x : i == 1 ? v4[1].y : i == 2 ? v4[1].z : v4[1].w;
            const uint32_t wc = i == 0 ? v4[2].x : i == 1 ? v4[2].y : i == 2 ? v4[2].z : v4[2].w;
            const uint32_t wd = i == 0 ? v4[3].x : i == 1 ? v4[3].y : i == 2 ? v4[3].z : v4[3].w;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t ab = __byte_perm(wa, wb, h ? 0x7362 : 0x5140);
              const uint32_t cd = __byte_perm(wc, wd, h ? 0x7362 : 0x5140);
              const uint32_t a0 = f16_lo(ab), a1 = f16_hi(ab), a2 = f16_lo(cd), a3 = f16_hi(cd);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16816(o[nb][2 * i + h], a0, a1, a2, a3, p[nb][0], p[nb][1]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.empty[ring.s]));
        }
        if (!live) break;
        // o[nb][d]: channels 16 g8 + 2 d (elements 0, 1) and + 1 (2, 3), rows 2 t4, 2 t4 + 1
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float lt = l[nb][h];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) lt += __shfl_xor_sync(0xFFFFFFFFu, lt, off);
            const int n = 8 * nb + 2 * t4 + h;
            float *dst = &sh.o[warp][n][16 * g8];
#pragma unroll
            for (int d = 0; d < 8; d += 2)
              *reinterpret_cast<float4 *>(dst + 2 * d) = make_float4(
                  o[nb][d][h], o[nb][d][h + 2], o[nb][d + 1][h], o[nb][d + 1][h + 2]);
            if (g8 == 0) {
              sh.m[warp][n] = m[nb][h];
              sh.r[warp][n] = r[nb][h] == -INFINITY ? -INFINITY : r[nb][h] - kBias;
              sh.l[warp][n] = lt;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.joined));
        if (!wait(smem_u32(&sh.joined), join_ph)) {
          live = false;
          break;
        }
        const bool whole = g.whole();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int n = 8 * nb + (tid >> 4), c = (tid & 15) * 8;
          if (n >= g.nrows) continue;
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, sh.m[w][n]);
          const float base = M == -INFINITY ? 0.f : M;
          float L = 0.f, x[8] = {};
#pragma unroll
          for (int w = 0; w < kConsumers; ++w) {
            L += sh.l[w][n] * ex2(sh.m[w][n] - base);
            const float f = ex2(sh.r[w][n] - base);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] += sh.o[w][n][c + k] * f;
          }
          const int pr = g.r0 + n;
          if (whole) {
            const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] *= inv;
            store8(static_cast<T *>(a.out) +
                       ((long long)(g.q0 + pr / a.G) * a.Hq + g.kvh * a.G + pr % a.G) * kHeadDim +
                       c,
                   x);
          } else {
            const long long at = (long long)part_slot(g) * a.slot_rows + n;
            store8(a.part_o + at * kHeadDim + c, x);
            if (c == 0) {
              a.part_ml[2 * at] = M;
              a.part_ml[2 * at + 1] = L;
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

template <class T, int NB>
cudaError_t few_go(const ChunkArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, int ctas,
                   cudaStream_t st) {
  constexpr int bytes = (int)sizeof(Shared<NB>);
  static_assert(bytes <= (NB == 1 ? 113 : 227) * 1024, "shared memory");
  const cudaError_t e = cudaFuncSetAttribute(
      chunk_few_kernel<T, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_few_kernel<T, NB>, dim3(ctas), dim3(kThreads), bytes, st, a, tk, tv);
}

}  // namespace

cudaError_t launch_chunk_few(int dtype, int rows, const ChunkArgs &a, const CUtensorMap &tk,
                             const CUtensorMap &tv, int ctas, cudaStream_t st) {
  if (dtype == KV_F16)
    return rows == 8 ? few_go<__half, 1>(a, tk, tv, ctas, st)
                     : few_go<__half, 2>(a, tk, tv, ctas, st);
  return rows == 8 ? few_go<__nv_bfloat16, 1>(a, tk, tv, ctas, st)
                   : few_go<__nv_bfloat16, 2>(a, tk, tv, ctas, st);
}

}  // namespace kvs
