// kv_chunk_q4.cu -- chunk attention over the 4-bit cache for few rows per kv head (a decode
// step, a few proposed tokens), and for fp32 q.  kv_chunk.cuh has the formula and how the
// work is cut.
//
// A CTA is four warps, or eight for long contexts, which take 32 tokens each in turn: a warp
// copies its own codes, scales and powers (asynchronously, one step ahead, the block table's
// entries before that), has a softmax of its own, and waits for no other until the end of a
// segment, where their results are joined.  (A warp that copied for four others by TMA and bulk copies was what bounded
// small pages: six copies per page of 16 tokens.)
//
// What bounds it: 4 bits leave two instructions a byte of the cache.  16 tokens by 8 rows take
// some 390 of a warp's instructions, 130 of them to expand the nibbles.  One token over 8 x
// <= 65536, 64/8 heads, bf16: 102 us with the joining of parts, 470 MB, 4.6 TB/s; the issue
// slots are busy for 58% of the time, DRAM for 46%.  Sixteen warps an SM at 128 registers (twenty
// at 96 spill: 139 us); pages looked up step by step cost 4 us.
//
// The products are 16 x 8 x 16, units 8 rows, as in kv_chunk_few.cu:
//   S^T (16 tokens x 8 rows) = K Q^T: the products sum over the channels, in any order that
//     K and Q share.  A thread's 16 bytes of codes are 32 channels of a token; a word's
//     nibbles i and i + 4 lie in one half each of a register, so that one operation puts
//     them into the mantissas of two f16, and one fma makes c s / 256 of them, exactly.
//   O^T (128 channels x 8 rows) += V^T P^T: pairs of two tokens' elements, a byte of two
//     channels at a time.
// Power bytes stay outside: K's multiplies the scores; V's joins the weight's exponent, weight
// = 2^(z + e_v - R) with R the row's running maximum of z + e_v, next to m, that of z, for the
// softmax's sum.  Rows of q are scaled into f16 by a power of two per row (see
// kv_chunk_few.cu); fp32 rows, and their weights, are taken as two f16 terms.
#include <type_traits>

#include "kv_chunk.cuh"
#include "kv_launch.h"
#include "kv_q4.cuh"
#include "kv_umma.cuh"

namespace kvs {
namespace {

constexpr float kMoveAt = 8.f;  // the maxima move when a weight would exceed 2^8 ...
constexpr float kShift = 7.f;   // ... times 2^7, so that small weights keep their f16 bits
constexpr int kRows = 8;        // rows of a unit
constexpr int kStep = 32;       // tokens of a warp's step
constexpr int kTile = 64;       // tokens per KV tile: what the work is cut by

// A step's bytes in shared memory: [token][64] of K's codes under a swizzle of 16-byte
// chunks, the same of V's, [token][8] of K's and of V's scales, K's and V's powers.
constexpr int kVAt = kStep * kQ4Bytes, kGroupAt = 2 * kVAt, kPowerAt = kGroupAt + 2 * kStep * kQ4Scales;
constexpr int kSlot = (kPowerAt + 2 * kStep + 127) / 128 * 128;

// A CTA has kWarps warps, 4 or (16-bit data) 8; an SM sixteen, of fp32 q eight.
template <class T, int kWarps> struct Shape {
  static constexpr int kCtas = (sizeof(T) == 2 ? 16 : 8) / kWarps;  // per SM
  static constexpr int kSlots = sizeof(T) == 2 ? 2 : 3;
};
template <class T, int kWarps> struct Shared {
  alignas(128) uint8_t slot[kWarps][Shape<T, kWarps>::kSlots][kSlot];
  float o[kWarps][kRows][kHeadDim];  // per warp, at the end of a segment
  float m[kWarps][kRows], r[kWarps][kRows], l[kWarps][kRows];
  ChunkShare<8> share;
  int red[32];
};

__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2 *>(&x); }
__device__ __forceinline__ uint32_t as_word(__half2 x) { return *reinterpret_cast<uint32_t *>(&x); }

// The integers n = c + 8 of the low (odd: high) nibbles of bytes 0 and 2 of a word, less 8,
// times a 256th of their scales s: an e4m3 code seven bits up is s / 256 in f16, the least ones
// included.  n is put into the mantissa of 1024 + n (odd: 64 + n), and (1024 + n) t - 1032 t
// (odd: (64 + n) t - 72 t), in one fma, is exact: s is an integer of 8 to 15 times a power of
// two, 1032 * 15 has 11 bits and factors of two.
struct Factor {
  __half2 s, even, odd;  // t = s / 256, -1032 t, -72 t of the two
};
__device__ __forceinline__ Factor factor_of(uint32_t codes) {  // in bytes 0 and 2
  const __half2 t = as_half2(codes << 7);
  return Factor{t, __hmul2(t, as_half2(0xE408E408u)), __hmul2(t, as_half2(0xD480D480u))};
}
// (One operation for mask and exponent, as long as both are in registers: of two immediates
// the compiler makes two.  One token over 8 x 65536: 127 -> 110 us.)
struct Bits {
  uint32_t mask[2], one[2];
  __device__ __forceinline__ Bits() {
    asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(mask[0]));
    asm volatile("mov.b32 %0, 0x00F000F0;" : "=r"(mask[1]));
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(one[0]));
    asm volatile("mov.b32 %0, 0x54005400;" : "=r"(one[1]));
  }
  template <bool odd> __device__ __forceinline__ uint32_t pair(uint32_t w, const Factor &f) const {
    uint32_t n;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(n) : "r"(w), "r"(mask[odd]), "r"(one[odd]));
    return as_word(__hfma2(as_half2(n), f.s, odd ? f.odd : f.even));
  }
};
// Which of the first eight tokens of sixteen a row of the products is (and of the last
// eight): with chunk c of token t at c ^ ((t >> 1) & 3), rows in this order meet distinct
// banks both as K's 16-byte and as V's 8-byte reads.
__device__ __forceinline__ int token_of_row(int row) { return (0x65742130u >> (4 * row)) & 7; }
__device__ __forceinline__ int chunk_at(int token, int chunk) {
  return token * kQ4Bytes + ((chunk ^ ((token >> 1) & 3)) << 4);
}

template <int n> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

template <class T, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, Shape<T, kWarps>::kCtas)
    chunk_q4_kernel(const __grid_constant__ ChunkArgs a) {
  constexpr bool kTwo = sizeof(T) == 4;  // q and the weights in two terms
  constexpr int kTerms = kTwo ? 2 : 1, kSlots = Shape<T, kWarps>::kSlots;
  extern __shared__ __align__(128) uint8_t smem[];
  using Sh = Shared<T, kWarps>;
  Sh &sh = *reinterpret_cast<Sh *>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g8 = lane >> 2, t4 = lane & 3;  // row and column group of the fragments
  const int tg = token_of_row(g8);          // the token of row g8 (and + 8)
  const int ps_log2 = 31 - __clz(a.ps);
  pdl_wait();
  if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  share_init(a, kRows, kTile, &sh.share, sh.red);
  const Bits bits;
  uint8_t *const slots = &sh.slot[warp][0][0];

  for (;;) {
    __syncthreads();
    if (tid == 0) share_next(a, kRows, kTile, &sh.share);
    __syncthreads();
    const int nseg = sh.share.nseg;
    if (nseg == 0) break;

    // The warp's steps of the list, in order: of segment sg the steps step0 + warp + 4 i below
    // step1.  The copies run kSlots - 1 steps ahead.  The pages of up to sixteen steps of a
    // segment are looked up together, while the step before them is copied: lanes 2 i and 2 i + 1
    // have the rows of the cache where the first, second sixteen tokens of the i-th are; -1: none.
    int list_sg = -1, list_at = 0, list_end = 0;  // the next step to look up
    int batch = -1, batch_n = 0, batch_i = 0;
    auto look_up = [&](int &n) -> int {
      while (list_sg < nseg && list_at >= list_end) {
        if (++list_sg == nseg) break;
        const ChunkSeg &g = sh.share.seg[list_sg];
        list_at = g.tile_lo * (kTile / kStep) + warp;
        list_end = min(g.tile_hi * (kTile / kStep), (g.len - 1) / kStep + 1);
      }
      int y = -1;
      n = 16;
      if (list_sg < nseg) {
        const ChunkSeg &g = sh.share.seg[list_sg];
        n = min(16, (list_end - list_at + kWarps - 1) / kWarps);
        const int tok = (list_at + kWarps * (lane >> 1)) * kStep + 16 * (lane & 1);
        if ((lane >> 1) < n && tok < g.len) {
          const int ph = a.bt[(long long)g.b * a.maxP + (tok >> ps_log2)];
          if (ph >= 0 && ph < a.nphys) y = (ph * a.Hkv + g.kvh) * a.ps + (tok & (a.ps - 1));
          else if (tok + 16 > seen_from(a, g)) flag_error(a.status, KV_ERR_BOUNDS);
        }
        list_at += kWarps * n;
      }
      return y;
    };
    int next_n, next_batch = look_up(next_n);
    int fill = 0;
    // starts the copies of the next step; bit i: its i-th sixteen tokens are there
    auto start = [&]() -> uint32_t {
      if (batch_i == batch_n) {
        batch = next_batch;
        batch_n = next_n;
        batch_i = 0;
        next_batch = look_up(next_n);
      }
      // (sixteen tokens that are not there are copied from the cache's first, and not used)
      const int at0 = __shfl_sync(0xFFFFFFFFu, batch, 2 * batch_i);
      const int at1 = __shfl_sync(0xFFFFFFFFu, batch, 2 * batch_i + 1);
      const int y0 = max(at0, 0), y1 = max(at1, 0);
      const uint32_t ok = (at0 >= 0 ? 1u : 0u) | (at1 >= 0 ? 2u : 0u);
      ++batch_i;
      const uint32_t to = smem_u32(slots + fill * kSlot);
      fill = fill + 1 == kSlots ? 0 : fill + 1;
      if (ok) {
        const uint32_t dst = to + chunk_at(lane >> 2, lane & 3);  // (eight tokens further: the same chunk)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const long long from = (long long)(h ? y1 : y0) * kQ4Bytes + lane * 16;
          const uint8_t *k = static_cast<const uint8_t *>(a.k) + from;
          const uint8_t *v = static_cast<const uint8_t *>(a.v) + from;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            cp_async16(dst + (2 * h + i) * 8 * kQ4Bytes, k + i * 8 * kQ4Bytes);
            cp_async16(dst + kVAt + (2 * h + i) * 8 * kQ4Bytes, v + i * 8 * kQ4Bytes);
          }
        }
        // scales: lanes 0 .. 15 K's, the others V's, eight lanes a half; powers: lanes 0 .. 3
        const int row = lane & 8 ? y1 : y0, last = lane & 1 ? y1 : y0;
        cp_async16(to + kGroupAt + lane * 16,
                   (lane & 16 ? a.v_group : a.k_group) + (long long)row * kQ4Scales + (lane & 7) * 16);
        if (lane < 4)
          cp_async16(to + kPowerAt + lane * 16, (lane & 2 ? a.v_scale : a.k_scale) + last);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      return ok;
    };
    uint32_t there[kSlots];  // of the steps in flight
#pragma unroll
    for (int i = 0; i + 1 < kSlots; ++i) there[i] = start();
    int drain = 0;

    for (int sg = 0; sg < nseg; ++sg) {
      const ChunkSeg g = sh.share.seg[sg];
      // Q: row n = g8, the 32 channels 32 t4 .. of K's rows that this thread reads, in the
      // pairs that a word's nibbles make
      uint32_t q[kTerms][16];
      float qf[2];  // scale * log2(e) / the row's power of two, rows 2 t4 and + 1
      int tq[2];    // their tokens
      {
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = 0.f;
        if (g8 < g.nrows) {
          const T *src = static_cast<const T *>(a.q) + row_offset(a, g.q0, g.kvh, g.r0 + g8);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float y[8];
            load8(src + 32 * t4 + 8 * i, y);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[8 * i + k] = y[k];
          }
        }
        float f = a.scale_log2;
        if constexpr (!std::is_same<T, __half>::value) {
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
          const int lo = 8 * (i >> 2) + (i & 3), hi = lo + 4;
          q[0][i] = pack2(x[lo], x[hi], __half{});
          if constexpr (kTwo) {
            const float2 h = unpack2(q[0][i], __half{});
            q[1][i] = pack2(x[lo] - h.x, x[hi] - h.y, __half{});
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          qf[h] = 256.f * __shfl_sync(0xFFFFFFFFu, f, 4 * (2 * t4 + h));  // (K's values are 256ths)
          tq[h] = g.len - g.n + token_of(a, g.r0 + min(2 * t4 + h, g.nrows - 1));
        }
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
      float bm[2] = {0.f, 0.f}, br[2] = {0.f, 0.f};  // the maxima that the weights refer to
      bool begun = false;                            // every row has seen a token
      const int end = min(g.tile_hi * (kTile / kStep), (g.len - 1) / kStep + 1);
      for (int step = g.tile_lo * (kTile / kStep) + warp; step < end; step += kWarps) {
        __syncwarp();  // the slot that is filled next has been read
        there[kSlots - 1] = start();
        cp_async_wait<kSlots - 1>();
        __syncwarp();  // (every lane's copies)
        const uint32_t have = there[0];
#pragma unroll
        for (int i = 0; i + 1 < kSlots; ++i) there[i] = there[i + 1];
        const uint8_t *slot = slots + drain * kSlot;
        drain = drain + 1 == kSlots ? 0 : drain + 1;
        const int tok0 = step * kStep;
        // every row sees all 32 tokens
        const bool clear = have == 3 && tok0 + 31 <= g.t_first &&
                           (a.window <= 0 || tok0 > g.t_last - a.window);
        // log2 of the weights in the sum and in the product; element i: token tg + 8 (i >> 1),
        // row 2 t4 + (i & 1)
        float e1[2][4], e2[2][4];
        uint32_t vb[2][2];  // V's power bytes
        const uint8_t *kc = slot + chunk_at(tg, t4);
        const uint8_t *kg = slot + kGroupAt + tg * kQ4Scales + 2 * t4, *kp = slot + kPowerAt + tg;
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          const uint4 u = *reinterpret_cast<const uint4 *>(kc + sub * 16 * kQ4Bytes);
          const uint4 v = *reinterpret_cast<const uint4 *>(kc + (sub * 16 + 8) * kQ4Bytes);
          const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
          // two scales of token tg, of token tg + 8
          const uint32_t g0 = *reinterpret_cast<const uint16_t *>(kg + sub * 16 * kQ4Scales);
          const uint32_t g1 = *reinterpret_cast<const uint16_t *>(kg + (sub * 16 + 8) * kQ4Scales);
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 2; ++c) {  // 16 channels, two words
            const Factor f0 = factor_of(__byte_perm(g0, 0, c ? 0x4141 : 0x4040));
            const Factor f1 = factor_of(__byte_perm(g1, 0, c ? 0x4141 : 0x4040));
#pragma unroll
            for (int j = 2 * c; j < 2 * c + 2; ++j) {
              const uint32_t a0 = bits.pair<0>(uu[j], f0), a1 = bits.pair<0>(vv[j], f1);
              const uint32_t a2 = bits.pair<1>(uu[j], f0), a3 = bits.pair<1>(vv[j], f1);
              const uint32_t b0 = bits.pair<0>(uu[j] >> 8, f0), b1 = bits.pair<0>(vv[j] >> 8, f1);
              const uint32_t b2 = bits.pair<1>(uu[j] >> 8, f0), b3 = bits.pair<1>(vv[j] >> 8, f1);
#pragma unroll
              for (int e = kTerms - 1; e >= 0; --e) {  // the small term first
                mma16816(s, a0, a1, a2, a3, q[e][4 * j], q[e][4 * j + 1]);
                mma16816(s, b0, b1, b2, b3, q[e][4 * j + 2], q[e][4 * j + 3]);
              }
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            // (power 255 gives infinity here, and a NaN vector's scales are 0: NaN)
            const float kf = __uint_as_float((uint32_t)kp[sub * 16 + 8 * k] << 23);
            vb[sub][k] = kp[kStep + sub * 16 + 8 * k];
            // vb - 127, in the mantissa of 2^23 + vb
            const float ev = __uint_as_float(0x4B000000u | vb[sub][k]) - 8388735.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x = s[2 * k + h] * kf;
              e1[sub][2 * k + h] = fmaf(x, qf[h], -bm[h]);
              e2[sub][2 * k + h] = fmaf(x, qf[h], ev - br[h]);
            }
          }
        }
        const uint32_t top = max(max(vb[0][0], vb[0][1]), max(vb[1][0], vb[1][1]));
        float over1 = e1[0][0], over2 = e2[0][0];
#pragma unroll
        for (int i = 1; i < 7; i += 2) {
          over1 = max3(over1, e1[i >> 2][i & 3], e1[(i + 1) >> 2][(i + 1) & 3]);
          over2 = max3(over2, e2[i >> 2][i & 3], e2[(i + 1) >> 2][(i + 1) & 3]);
        }
        over1 = fmaxf(over1, e1[1][3]);
        over2 = fmaxf(over2, e2[1][3]);
        // bit 4 row + k + 2 sub: row + 8 k of the products has a V to be cleared
        uint32_t bad = 0;
        const bool rare = over1 > kMoveAt || over2 > kMoveAt + kShift || top == (uint32_t)kQ4NanPower;
        if (__any_sync(0xFFFFFFFFu, rare) || !clear || !begun) {
          // tokens that are not seen, NaN vectors, and maxima that move
          begun = true;
#pragma unroll
          for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int pos = tok0 + 16 * sub + tg + 8 * k;
              const bool token = ((have >> sub) & 1) && pos < g.len;
              const bool nan = vb[sub][k] == (uint32_t)kQ4NanPower;
              bad |= __ballot_sync(0xFFFFFFFFu, (!token || nan) && t4 == k + 2 * sub);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float &z = e1[sub][2 * k + h], &y = e2[sub][2 * k + h];
                const bool see = token && pos <= tq[h] && (a.window <= 0 || pos - tq[h] > -a.window);
                z = see ? z + bm[h] : -INFINITY;
                y = !see ? -INFINITY : nan ? __uint_as_float(0x7FC00000u) : y + br[h];
              }
            }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float mz = fmaxf(fmaxf(e1[0][h], e1[0][h + 2]), fmaxf(e1[1][h], e1[1][h + 2]));
            float my = fmaxf(fmaxf(e2[0][h], e2[0][h + 2]), fmaxf(e2[1][h], e2[1][h + 2]));
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              mz = fmaxf(mz, __shfl_xor_sync(0xFFFFFFFFu, mz, off));
              my = fmaxf(my, __shfl_xor_sync(0xFFFFFFFFu, my, off));
            }
            mz = fmaxf(mz, m[h]);
            my = fmaxf(my, r[h]);
            // (from -inf: 0, and 1 where it stays there)
            const float al = mz == -INFINITY ? 1.f : ex2(m[h] - mz);
            const float ao = my == -INFINITY ? 1.f : ex2(r[h] - my);
            m[h] = mz;
            r[h] = my;
            bm[h] = mz == -INFINITY ? 0.f : mz;
            br[h] = my == -INFINITY ? 0.f : my - kShift;
            begun &= mz != -INFINITY && my != -INFINITY;
            l[h] *= al;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              o[d][h] *= ao;
              o[d][h + 2] *= ao;
            }
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
#pragma unroll
              for (int i = h; i < 4; i += 2) {
                e1[sub][i] -= bm[h];
                e2[sub][i] -= br[h];
              }
          }
          begun = __all_sync(0xFFFFFFFFu, begun);
        }
        // O^T: rows 2 t4, 2 t4 + 1 (+ 8) of the products; channels 16 g8 .. + 15
        const int ta = token_of_row(2 * t4), tb = token_of_row(2 * t4 + 1);
        const uint8_t *va = slot + kVAt + chunk_at(ta, g8 >> 1) + 8 * (g8 & 1);
        const uint8_t *vc = slot + kVAt + chunk_at(tb, g8 >> 1) + 8 * (g8 & 1);
        const uint8_t *vg = slot + kGroupAt + kStep * kQ4Scales + g8;
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            l[i & 1] += ex2(e1[sub][i]);
            w[i] = ex2(e2[sub][i]);
          }
          uint32_t p[kTerms][2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t hi = pack2(w[2 * k], w[2 * k + 1], __half{});
            p[0][k] = movm_t(hi);
            if constexpr (kTwo) {
              const float2 h = unpack2(hi, __half{});
              p[1][k] = movm_t(pack2(w[2 * k] - h.x, w[2 * k + 1] - h.y, __half{}));
            }
          }
          uint2 v2[4];
          uint32_t sb[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v2[i] = *reinterpret_cast<const uint2 *>((i & 1 ? vc : va) + (sub * 16 + 8 * (i >> 1)) * kQ4Bytes);
            sb[i] = vg[(sub * 16 + 8 * (i >> 1) + (i & 1 ? tb : ta)) * kQ4Scales];
          }
          // rows without a token and NaN vectors must not meet a weight of 0: their scales
          // are cleared (a row that sees a NaN vector has a NaN weight)
          if (bad) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((bad >> (4 * (2 * t4 + (i & 1)) + (i >> 1) + 2 * sub)) & 1) sb[i] = 0;
          }
          const Factor f0 = factor_of(sb[0] | (sb[1] << 16));
          const Factor f1 = factor_of(sb[2] | (sb[3] << 16));
#pragma unroll
          for (int d = 0; d < 8; ++d) {  // a byte of two channels: a block of O^T
            const int byte = 0x0400 + 0x0101 * (d & 3);
            const uint32_t x = __byte_perm(d < 4 ? v2[0].x : v2[0].y, d < 4 ? v2[1].x : v2[1].y, byte);
            const uint32_t y = __byte_perm(d < 4 ? v2[2].x : v2[2].y, d < 4 ? v2[3].x : v2[3].y, byte);
            const uint32_t a0 = bits.pair<0>(x, f0), a1 = bits.pair<1>(x, f0);
            const uint32_t a2 = bits.pair<0>(y, f1), a3 = bits.pair<1>(y, f1);
            if constexpr (kTwo) {
              float t[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816(t, a0, a1, a2, a3, p[1][0], p[1][1]);
              mma16816(t, a0, a1, a2, a3, p[0][0], p[0][1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) o[d][i] += t[i];
            } else {
              mma16816(o[d], a0, a1, a2, a3, p[0][0], p[0][1]);
            }
          }
        }
      }
      // elements 0, 1 of o[d]: channel 16 g8 + 2 d, rows 2 t4 and 2 t4 + 1; 2, 3: the next one
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float lt = l[h];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) lt += __shfl_xor_sync(0xFFFFFFFFu, lt, off);
        const int n = 2 * t4 + h;
#pragma unroll
        for (int d = 0; d < 8; d += 2)
          *reinterpret_cast<float4 *>(&sh.o[warp][n][16 * g8 + 2 * d]) =
              make_float4(o[d][h], o[d][h + 2], o[d + 1][h], o[d + 1][h + 2]);
        if (g8 == 0) {
          sh.m[warp][n] = m[h];
          sh.r[warp][n] = r[h] == -INFINITY ? -INFINITY : r[h] - kShift + 8.f;  // (V's are 256ths)
          sh.l[warp][n] = lt;
        }
      }
      __syncthreads();
      const bool whole = g.whole();
      for (int n = tid >> 4; n < min(kRows, g.nrows); n += 2 * kWarps) {
        const int c = (tid & 15) * 8;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh.m[w][n]);
        const float base = top == -INFINITY ? 0.f : top;
        // (the factors carry V's powers, 2^-110 and up: without 2^64 those of warps whose
        // maximum is 2^-9 below the row's would be 0)
        constexpr float kUp = 64.f, kDown = 0x1p-64f;
        float sum = 0.f, x[8] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          sum += sh.l[w][n] * ex2(sh.m[w][n] - base);
          const float f = ex2(sh.r[w][n] - base + kUp);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] += sh.o[w][n][c + k] * f;
        }
        const int pr = g.r0 + n;
        if (whole) {
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
      __syncthreads();
    }
    cp_async_wait<0>();
  }
}

template <class T, int kWarps> cudaError_t q4_go(const ChunkArgs &a, int ctas, cudaStream_t st) {
  constexpr int bytes = (int)sizeof(Shared<T, kWarps>);
  static_assert(bytes <= (228 / Shape<T, kWarps>::kCtas - 1) * 1024, "shared memory");
  const cudaError_t e = cudaFuncSetAttribute(
      chunk_q4_kernel<T, kWarps>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_q4_kernel<T, kWarps>, dim3(ctas), dim3(32 * kWarps), bytes, st, a);
}

}  // namespace

FewShape chunk_q4_shape(int dtype, bool eight) {
  return FewShape{kRows, kTile, dtype == KV_F32 ? Shape<float, 4>::kCtas
                                : eight         ? Shape<__half, 8>::kCtas
                                                : Shape<__half, 4>::kCtas};
}

cudaError_t launch_chunk_q4(int dtype, bool eight, const ChunkArgs &a, int ctas, cudaStream_t st) {
  if (dtype == KV_F32) return q4_go<float, 4>(a, ctas, st);
  if (dtype == KV_F16) return eight ? q4_go<__half, 8>(a, ctas, st) : q4_go<__half, 4>(a, ctas, st);
  return eight ? q4_go<__nv_bfloat16, 8>(a, ctas, st) : q4_go<__nv_bfloat16, 4>(a, ctas, st);
}

}  // namespace kvs
