// kv_chunk.cu -- chunk attention on the CUDA cores in fp32, and the combine
// of partial results.  kv_chunk.cuh has the formula and how the work is cut.
#include <algorithm>
#include <type_traits>

#include "kv_chunk.cuh"
#include "kv_launch.h"
#include "kv_q8.cuh"

namespace kvs {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;             // tokens per KV tile
constexpr int kQStr = kHeadDim + 4;   // padded rows: 16-byte reads of 16 rows meet distinct banks
constexpr int kPStr = kTile + 4;

// Units of 64 rows.  256 threads as 16 x 16: thread (ty, tx) holds rows
// 4 ty .. + 3; of the scores the columns tx + 16 j, of the output
// the channels 4 tx .. + 3 and 64 + 4 tx .. + 3.  Per tile: scores = Q K^T
// (a 4 x 4 register block per thread), one streaming-softmax step (row
// maximum and sum over the 16 tx lanes), output += P V.  The weights P take
// K's place in shared memory once the scores are done, so that two CTAs fit an
// SM.  FP32 multiply-adds and the shared-memory reads that feed them bound it: 256
// rows over 8192 tokens, 32/8 heads, 875 us on one GB300, 38.7 TFLOP/s (two products
// per instruction, with the sums over even and odd channels apart, 978 us).
constexpr int MR = 4;
constexpr int kTileRows = 16 * MR;
constexpr int kKBytes = kTile * kQStr * 4;
constexpr int kTileSmem = kTileRows * kQStr * 4 + kKBytes + kTile * kHeadDim * 4;
static_assert(kTileRows * kPStr * 4 <= kKBytes, "P takes K's place");

// A row's running result: log2-domain maximum, sum, and four channels.
struct Joined {
  float m, l;
  float4 o;
};
__device__ __forceinline__ void join_one(Joined &a, float m, float l, const float4 &o) {
  const float M = fmaxf(a.m, m), base = M == -INFINITY ? 0.f : M;
  const float f = ex2(a.m - base), h = ex2(m - base);
  a.m = M;
  a.l = a.l * f + l * h;
  a.o = make_float4(a.o.x * f + o.x * h, a.o.y * f + o.y * h, a.o.z * f + o.z * h,
                    a.o.w * f + o.w * h);
}
// Four channels from c on of a row at token t, whose weights' sum is l: the infinities and
// NaN it sees among them in V of type T, in KV tiles [lo, hi), where its result is not
// finite.  (A result over the 8-bit cache stays: codes have no infinity, and a NaN vector
// is NaN in every channel.)
template <class T>
__device__ __forceinline__ void put_odd(const ChunkArgs &a, int b, int kvh, int t, int c, int lo,
                                        int hi, int tile, float l, float4 &x) {
  if (finite(x) || l != l) return;
  const Seen s = seen_tokens(a, t, lo, hi, tile);
  const Odd odd = odd_values<T, 4>(a, b, kvh, s.lo, s.hi, c);
  if (odd.any(0)) x.x = odd.sum(0);
  if (odd.any(1)) x.y = odd.sum(1);
  if (odd.any(2)) x.z = odd.sum(2);
  if (odd.any(3)) x.w = odd.sum(3);
}
template <class T>
__device__ __forceinline__ void join_store(const ChunkArgs &a, const int4 &u, int q0, int r,
                                           int lane, const Joined &x) {
  const float inv = x.l == 0.f ? 0.f : 1.f / x.l;
  T *dst = static_cast<T *>(a.out) + row_offset(a, q0, u.y, u.z + r) + lane * 4;
  if constexpr (std::is_same_v<T, float>)
    *reinterpret_cast<float4 *>(dst) =
        make_float4(x.o.x * inv, x.o.y * inv, x.o.z * inv, x.o.w * inv);
  else
    *reinterpret_cast<uint2 *>(dst) =
        make_uint2(pack2(x.o.x * inv, x.o.y * inv, T{}), pack2(x.o.z * inv, x.o.w * inv, T{}));
}
// A weight of a token that the row does not see is -0: it must not meet an infinity or
// NaN of V.  One that the row sees may be 0.
__device__ __forceinline__ bool unseen(float weight) { return __float_as_uint(weight) == 0x80000000u; }

// 4 channels (of lane `lane`) of one cached vector in fp32
template <bool Q8>
__device__ __forceinline__ float4 cached4(const void *base, const uint8_t *scale, long long vec,
                                          int lane) {
  if constexpr (Q8) {
    float x[4];
    q8_unpack4(reinterpret_cast<const uint32_t *>(base)[vec * (kHeadDim / 4) + lane], x);
    const float s = q8_scale(scale[vec]);
    return make_float4(x[0] * s, x[1] * s, x[2] * s, x[3] * s);
  } else {
    return reinterpret_cast<const float4 *>(base)[vec * (kHeadDim / 4) + lane];
  }
}

// 8 channels of one cached vector in fp32
template <bool Q8>
__device__ __forceinline__ void cached8(const void *base, const uint8_t *scale, long long vec,
                                        int c, float (&x)[8]) {
  if constexpr (Q8) {
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(base) +
                                                     vec * kHeadDim + c);
    float lo[4], hi[4];
    q8_unpack4(w.x, lo);
    q8_unpack4(w.y, hi);
    const float s = q8_scale(scale[vec]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = lo[i] * s;
      x[4 + i] = hi[i] * s;
    }
  } else {
    load8(static_cast<const float *>(base) + vec * kHeadDim + c, x);
  }
}

template <bool Q8>
__global__ void __launch_bounds__(kThreads) chunk_core_kernel(const __grid_constant__ ChunkArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ ChunkShare<16> share;
  __shared__ int red[32];
  __shared__ int tok_ok[kTile];
  float *Qs = reinterpret_cast<float *>(smem);
  float *Ks = Qs + kTileRows * kQStr;
  float *Vs = Ks + kTile * kQStr;
  float *Ps = Ks;
  pdl_wait();
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int ps_log2 = 31 - __clz(a.ps);
  if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  share_init(a, kTileRows, kTile, &share, red);
  for (;;) {
    __syncthreads();
    if (tid == 0) share_next(a, kTileRows, kTile, &share);
    __syncthreads();
    if (share.nseg == 0) break;
    for (int sg = 0; sg < share.nseg; ++sg) {
      const ChunkSeg g = share.seg[sg];
      __syncthreads();  // the previous segment's Q is read
      for (int i = tid; i < kTileRows * 16; i += kThreads) {
        const int r = i >> 4, c = (i & 15) * 8;
        float x[8] = {};
        if (r < g.nrows) {
          load8(static_cast<const float *>(a.q) + row_offset(a, g.q0, g.kvh, g.r0 + r) + c, x);
        }
        store8(Qs + r * kQStr + c, x);
      }
      int t[MR];
      float m[MR], l[MR], o[MR][8];
#pragma unroll
      for (int r = 0; r < MR; ++r) {
        t[r] = g.len - g.n + token_of(a, g.r0 + min(ty * MR + r, g.nrows - 1));
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) o[r][c] = 0.f;
      }
      // the pages of this thread's tokens of a tile (-1: none, or one that no row
      // sees; -2: out of range), looked up a tile ahead
      const int from = seen_from(a, g);
      constexpr int kLoads = kTile * 16 / kThreads;
      int ph[kLoads];
      auto look_up = [&](int tile) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int pos = tile * kTile + (tid >> 4) + k * (kThreads / 16);
          ph[k] = -1;
          if (tile < g.tile_hi && pos < g.len) {
            const int p = a.bt[(long long)g.b * a.maxP + (pos >> ps_log2)];
            ph[k] = p >= 0 && p < a.nphys ? p : pos >= from ? -2 : -1;
          }
        }
      };
      look_up(g.tile_lo);
      for (int tile = g.tile_lo; tile < g.tile_hi; ++tile) {
        const int tok0 = tile * kTile;
        // K and V of the tile; tokens past the end or of a bad page are zero
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int tok = (tid >> 4) + k * (kThreads / 16), c = (tid & 15) * 8;
          float kx[8] = {}, vx[8] = {};
          const bool ok = ph[k] >= 0;
          if (ok) {
            // (rows of the cache fit int32)
            const int vec = (ph[k] * a.Hkv + g.kvh) * a.ps + ((tok0 + tok) & (a.ps - 1));
            cached8<Q8>(a.k, a.k_scale, vec, c, kx);
            cached8<Q8>(a.v, a.v_scale, vec, c, vx);
          } else if (ph[k] == -2 && c == 0) {
            flag_error(a.status, KV_ERR_BOUNDS);
          }
          if (c == 0) tok_ok[tok] = ok;
          store8(Ks + tok * kQStr + c, kx);
          store8(Vs + tok * kHeadDim + c, vx);
        }
        look_up(tile + 1);
        __syncthreads();
        float s[MR][4] = {};
#pragma unroll 4
        for (int d = 0; d < kHeadDim; d += 4) {
          float4 qv[MR], kv[4];
#pragma unroll
          for (int r = 0; r < MR; ++r)
            qv[r] = *reinterpret_cast<const float4 *>(Qs + (ty * MR + r) * kQStr + d);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            kv[j] = *reinterpret_cast<const float4 *>(Ks + (tx + 16 * j) * kQStr + d);
#pragma unroll
          for (int r = 0; r < MR; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              s[r][j] += qv[r].x * kv[j].x + qv[r].y * kv[j].y + qv[r].z * kv[j].z +
                         qv[r].w * kv[j].w;
        }
        bool ok[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) ok[j] = tok_ok[tx + 16 * j];
        __syncthreads();  // every thread is done with K: P takes its place
#pragma unroll
        for (int r = 0; r < MR; ++r) {
          const int hi = vis_hi(t[r], tok0), lo = vis_lo(t[r], tok0, a.window);
          float mx = m[r];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = tx + 16 * j;
            s[r][j] = ok[j] && c <= hi && c >= lo ? s[r][j] * a.scale_log2 : -INFINITY;
            mx = fmaxf(mx, s[r][j]);
          }
#pragma unroll
          for (int off = 8; off > 0; off >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off, 16));
          const float base = mx == -INFINITY ? 0.f : mx;
          const float alpha = ex2(m[r] - base);
          m[r] = mx;
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p = s[r][j] == -INFINITY ? -0.f : ex2(s[r][j] - base);
            sum += p;
            Ps[(ty * MR + r) * kPStr + tx + 16 * j] = p;
          }
          l[r] = l[r] * alpha + sum;
#pragma unroll
          for (int c = 0; c < 8; ++c) o[r][c] *= alpha;
        }
        __syncthreads();
        // whether some row does not see some token
        const bool edge = tok0 + kTile - 1 > g.t_first || a.window > 0;
#pragma unroll 2
        for (int j0 = 0; j0 < kTile; j0 += 4) {
          // the weights of four tokens in one read (a read each kept the
          // shared-memory pipe as busy as the multiply-adds: 36 TFLOP/s)
          float pw[MR][4];
#pragma unroll
          for (int r = 0; r < MR; ++r) {
            const float4 w = *reinterpret_cast<const float4 *>(Ps + (ty * MR + r) * kPStr + j0);
            pw[r][0] = w.x;
            pw[r][1] = w.y;
            pw[r][2] = w.z;
            pw[r][3] = w.w;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float *v = Vs + (j0 + j) * kHeadDim + tx * 4;
            const float4 v0 = *reinterpret_cast<const float4 *>(v);
            const float4 v1 = *reinterpret_cast<const float4 *>(v + 64);
            const float vv[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int r = 0; r < MR; ++r) {
              if (edge && unseen(pw[r][j])) continue;
#pragma unroll
              for (int c = 0; c < 8; ++c) o[r][c] += pw[r][j] * vv[c];
            }
          }
        }
        __syncthreads();
      }
      const bool whole = g.whole();
      const int slot = part_slot(g);
#pragma unroll
      for (int r = 0; r < MR; ++r) {
        float sum = l[r];
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off, 16);
        const int rr = ty * MR + r;
        if (rr >= g.nrows) continue;
        float4 x0 = make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
        float4 x1 = make_float4(o[r][4], o[r][5], o[r][6], o[r][7]);
        if (whole) {
          if constexpr (!Q8) {
            put_odd<float>(a, g.b, g.kvh, t[r], tx * 4, g.tile_lo, g.tile_hi, kTile, sum, x0);
            put_odd<float>(a, g.b, g.kvh, t[r], 64 + tx * 4, g.tile_lo, g.tile_hi, kTile, sum, x1);
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          float *dst = static_cast<float *>(a.out) + row_offset(a, g.q0, g.kvh, g.r0 + rr);
          *reinterpret_cast<float4 *>(dst + tx * 4) =
              make_float4(x0.x * inv, x0.y * inv, x0.z * inv, x0.w * inv);
          *reinterpret_cast<float4 *>(dst + 64 + tx * 4) =
              make_float4(x1.x * inv, x1.y * inv, x1.z * inv, x1.w * inv);
        } else {
          const long long pr = (long long)slot * a.slot_rows + rr;
          float *dst = a.part_o + pr * kHeadDim + tx * 4;
          *reinterpret_cast<float4 *>(dst) = x0;
          *reinterpret_cast<float4 *>(dst + 64) = x1;
          if (tx == 0) {
            a.part_ml[2 * pr] = m[r];
            a.part_ml[2 * pr + 1] = sum;
          }
        }
      }
    }
  }
}

// Few rows: units of R = 4 or 8.  A warp takes 8 of a tile's 64 tokens, with a
// softmax of its own, and K and V go from memory to registers: lane l holds
// channels 4 l .. + 3 of the unit's q, of its output and of the token at hand.
// The 8 R partial dot products of eight tokens are summed over the lanes by
// halving exchanges (one shuffle per sum), which leaves lane l the rows
// (l & 3) R / 4 .. of token l / 4; the weights come back through shared memory.
// The K/V stream bounds it at one row per kv head; at 8, multiply-adds and
// shuffles about as much.  One token over 4 x 8192 tokens, 32/8 heads: 44 us on one
// GB300, 6.1 TB/s; 33 rows over 4096 tokens, one head: 13.6 us, the chain of a
// CTA's few tiles and the combine.
constexpr int kFewWarps = kThreads / 32;
constexpr float kMoveAt = 8.f;  // the maximum moves when a weight would exceed 2^8
template <int R> struct FewShared {
  float p[kFewWarps][8][R];  // weights of a warp's tokens
  float alpha[kFewWarps][R];
  float o[kFewWarps][R][kHeadDim];  // at the end of a segment
  float m[kFewWarps][R], l[kFewWarps][R];
  ChunkShare<16> share;
  int red[32];
};

template <int R, bool Q8>
__global__ void __launch_bounds__(kThreads, R == 4 ? 2 : 1)
    chunk_rows_kernel(const __grid_constant__ ChunkArgs a) {
  constexpr int L = R / 4;  // rows whose sums a lane ends up with
  extern __shared__ __align__(16) uint8_t smem[];
  FewShared<R> &sh = *reinterpret_cast<FewShared<R> *>(smem);
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ps_log2 = 31 - __clz(a.ps);
  const int tok = lane >> 2, row0 = (lane & 3) * L;
  if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  share_init(a, R, kTile, &sh.share, sh.red);
  for (;;) {
    __syncthreads();
    if (tid == 0) share_next(a, R, kTile, &sh.share);
    __syncthreads();
    if (sh.share.nseg == 0) break;
    for (int sg = 0; sg < sh.share.nseg; ++sg) {
      const ChunkSeg g = sh.share.seg[sg];
      float4 q[R], o[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        o[r] = q[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < g.nrows) {
          q[r] = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) +
                                                   row_offset(a, g.q0, g.kvh, g.r0 + r) + 4 * lane);
        }
      }
      int t[L];
      float m[L], l[L];
#pragma unroll
      for (int i = 0; i < L; ++i) {
        t[i] = g.len - g.n + token_of(a, g.r0 + min(row0 + i, g.nrows - 1));
        m[i] = -INFINITY;
        l[i] = 0.f;
      }
      // page of this warp's eight tokens of a tile, a tile ahead (as above)
      const int from = seen_from(a, g);
      auto look_up = [&](int tile) -> int {
        const int pos = tile * kTile + warp * 8;
        if (tile >= g.tile_hi || pos >= g.len) return -1;
        const int ph = a.bt[(long long)g.b * a.maxP + (pos >> ps_log2)];
        return ph >= 0 && ph < a.nphys ? ph : pos + 8 > from ? -2 : -1;
      };
      int next = look_up(g.tile_lo);
      for (int tile = g.tile_lo; tile < g.tile_hi; ++tile) {
        const int ph = next, pos0 = tile * kTile + warp * 8;
        next = look_up(tile + 1);
        if (ph < 0) {  // no token that a row sees, or a bad page
          if (ph == -2 && lane == 0) flag_error(a.status, KV_ERR_BOUNDS);
          continue;
        }
        const int count = min(8, g.len - pos0);
        // (rows of the cache fit int32)
        const int vec0 = (ph * a.Hkv + g.kvh) * a.ps + (pos0 & (a.ps - 1));
        float4 kx[8], vx[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          kx[j] = vx[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (j < count) {
            kx[j] = cached4<Q8>(a.k, a.k_scale, vec0 + j, lane);
            vx[j] = cached4<Q8>(a.v, a.v_scale, vec0 + j, lane);
          }
        }
        float s[8 * R];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int r = 0; r < R; ++r)
            s[j * R + r] = q[r].x * kx[j].x + q[r].y * kx[j].y + q[r].z * kx[j].z +
                           q[r].w * kx[j].w;
#pragma unroll
        for (int off = 16, n = 8 * R; off > 0; off >>= 1, n >>= 1) {
          const bool up = lane & off;
#pragma unroll
          for (int i = 0; i < n / 2; ++i) {
            const float give = up ? s[i] : s[i + n / 2], keep = up ? s[i + n / 2] : s[i];
            s[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, off);
          }
        }
        const int pos = pos0 + tok;
        bool move = false;
#pragma unroll
        for (int i = 0; i < L; ++i) {
          const bool see = tok < count && pos <= t[i] &&
                           (a.window <= 0 || pos - t[i] > -a.window);
          s[i] = see ? s[i] * a.scale_log2 : -INFINITY;
          move |= s[i] > m[i] + kMoveAt;
        }
        if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
          for (int i = 0; i < L; ++i) {
            float mx = s[i];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
              mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
            mx = fmaxf(mx, m[i]);
            const float f = mx == -INFINITY ? 1.f : ex2(m[i] - mx);
            m[i] = mx;
            l[i] *= f;
            if (tok == 0) sh.alpha[warp][row0 + i] = f;
          }
          __syncwarp();
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float f = sh.alpha[warp][r];
            o[r] = make_float4(o[r].x * f, o[r].y * f, o[r].z * f, o[r].w * f);
          }
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
          const float p =
              s[i] == -INFINITY ? -0.f : ex2(s[i] - (m[i] == -INFINITY ? 0.f : m[i]));
          l[i] += p;
          sh.p[warp][tok][row0 + i] = p;
        }
        __syncwarp();
        // whether some row does not see some token
        const bool edge = pos0 + 7 > g.t_first || a.window > 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
          for (int r0 = 0; r0 < R; r0 += 4) {
            const float4 w = *reinterpret_cast<const float4 *>(&sh.p[warp][j][r0]);
            const float ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if (edge && unseen(ww[r])) continue;
              float4 &x = o[r0 + r];
              x = make_float4(x.x + ww[r] * vx[j].x, x.y + ww[r] * vx[j].y, x.z + ww[r] * vx[j].z,
                              x.w + ww[r] * vx[j].w);
            }
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
        *reinterpret_cast<float4 *>(&sh.o[warp][r][4 * lane]) = o[r];
#pragma unroll
      for (int i = 0; i < L; ++i) {
        float sum = l[i];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
        if (tok == 0) {
          sh.m[warp][row0 + i] = m[i];
          sh.l[warp][row0 + i] = sum;
        }
      }
      __syncthreads();
      // a warp joins a row (of 4 rows: half the warps), a lane four channels
      if (warp < g.nrows) {
        const int r = warp;
        Joined x{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w)
          join_one(x, sh.m[w][r], sh.l[w][r],
                   *reinterpret_cast<const float4 *>(&sh.o[w][r][4 * lane]));
        if (g.whole()) {
          if constexpr (!Q8)
            put_odd<float>(a, g.b, g.kvh, g.len - g.n + token_of(a, g.r0 + r), 4 * lane, g.tile_lo,
                           g.tile_hi, kTile, x.l, x.o);
          join_store<float>(a, make_int4(g.b, g.kvh, g.r0, g.nrows), g.q0, r, lane, x);
        } else {
          const long long at = (long long)part_slot(g) * a.slot_rows + r;
          *reinterpret_cast<float4 *>(a.part_o + at * kHeadDim + 4 * lane) = x.o;
          if (lane == 0) {
            a.part_ml[2 * at] = x.m;
            a.part_ml[2 * at + 1] = x.l;
          }
        }
      }
      __syncthreads();
    }
  }
}

// Joins the parts of every unit that several CTAs share: CTA i of the
// attention left part 2 i + 1, the CTAs i + 1 .. j parts 2 (i + 1) .. 2 j.  A
// lane takes four channels, a warp four rows, so that the loads of four rows
// are in flight together (one row at a time took three times as long).  Few
// parts: each warp joins all parts of its rows (of one, when there are no more
// rows than that).  Many (a long context and few rows): the block's warps share
// the parts of four rows, or of one, when there are blocks enough (8 rows of one kv
// head over 30000 tokens, 304 parts: the call 25 -> 15.5 us).
constexpr int kJoinRows = 4;
// rows r0 .. r0 + R - 1 of the parts of the CTAs from, from + step, .. up to `last`, U of
// them in flight
template <int R, int U>
__device__ __forceinline__ void join_rows(const ChunkArgs &a, int first, int last, int from,
                                          int step, int r0, int nrows, int lane,
                                          Joined (&acc)[R]) {
#pragma unroll
  for (int i = 0; i < R; ++i)
    acc[i] = Joined{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 1
  for (int j0 = from; j0 <= last; j0 += step * U) {
    float2 ml[U][R];
    float4 o[U][R];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int j = j0 + k * step;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        ml[k][i] = make_float2(-INFINITY, 0.f);
        o[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j <= last) {
          const long long row = (long long)(j == first ? 2 * j + 1 : 2 * j) * a.slot_rows + r0 +
                                min(i, nrows - 1 - r0);
          ml[k][i] = *reinterpret_cast<const float2 *>(a.part_ml + 2 * row);
          o[k][i] = *reinterpret_cast<const float4 *>(a.part_o + row * kHeadDim + lane * 4);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int i = 0; i < R; ++i) join_one(acc[i], ml[k][i].x, ml[k][i].y, o[k][i]);
  }
}
// join_store, and whether the result is not finite: such channels are infinities until
// mend_rows has read the cache again (NaN stays where the row's weights are).
template <class T>
__device__ __forceinline__ bool combine_store(const ChunkArgs &a, const int4 &u, int q0, int r,
                                              int lane, Joined x) {
  const bool odd = !finite(x.o) && x.l == x.l && !a.k_scale;
  if (odd) {
    x.o.x = finite(x.o.x) ? x.o.x : INFINITY;
    x.o.y = finite(x.o.y) ? x.o.y : INFINITY;
    x.o.z = finite(x.o.z) ? x.o.z : INFINITY;
    x.o.w = finite(x.o.w) ? x.o.w : INFINITY;
  }
  join_store<T>(a, u, q0, r, lane, x);
  return odd;
}
// Rows r .. r + count - 1 of the unit, and so on every `step` rows, all written by this
// thread: put_odd for what combine_store left.  At the kernel's end, by itself: in
// combine_store it cost the registers of the loads in flight (8 rows over 32k tokens in
// 8 bits 86 -> 96 us).
template <class T>
__device__ __noinline__ void mend_rows(const ChunkArgs &a, int4 u, int q0, int r, int step, int count,
                                       int lane) {
  const int t0 = a.ctx[u.x] - (a.q_start[u.x + 1] - q0);
  for (; r < u.w; r += step)
    for (int i = r; i < min(r + count, u.w); ++i) {
      T *dst = static_cast<T *>(a.out) + row_offset(a, q0, u.y, u.z + i) + 4 * lane;
      float x[4];
      load_n(dst, x);
      if (finite(make_float4(x[0], x[1], x[2], x[3]))) continue;
      const Seen s = seen_tokens(a, t0 + token_of(a, u.z + i), 0, INT_MAX, 1);
      const Odd odd = odd_values<T, 4>(a, u.x, u.y, s.lo, s.hi, 4 * lane);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (odd.any(k) && x[k] == INFINITY) dst[k] = (T)odd.sum(k);
    }
}
template <class T>
__global__ void __launch_bounds__(256) chunk_combine_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ Joined part[8][kJoinRows][32];
  pdl_wait();
  const int4 u = a.meta[2 * blockIdx.x], w = a.meta[2 * blockIdx.x + 1];
  if (u.x < 0) return;
  const int first = blockIdx.x, last = w.y, nrows = u.w;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool odd = false;
  int from, step, count = 1;  // the rows this thread writes
  if (last - first < 8 && nrows <= 8 * (int)gridDim.y) {
    from = blockIdx.y * 8 + warp;
    step = nrows;
    if (from >= nrows) return;
    Joined one[1];
    join_rows<1, 8>(a, first, last, first, 1, from, nrows, lane, one);
    odd = combine_store<T>(a, u, w.x, from, lane, one[0]);
  } else if (last - first < 8) {
    Joined acc[kJoinRows];
    from = (blockIdx.y * 8 + warp) * kJoinRows;
    step = gridDim.y * 8 * kJoinRows;
    count = kJoinRows;
    for (int r0 = from; r0 < nrows; r0 += step) {
      join_rows<kJoinRows, 2>(a, first, last, first, 1, r0, nrows, lane, acc);
#pragma unroll
      for (int i = 0; i < kJoinRows; ++i)
        if (r0 + i < nrows) odd |= combine_store<T>(a, u, w.x, r0 + i, lane, acc[i]);
    }
  } else {
    const int per = nrows <= (int)gridDim.y ? 1 : kJoinRows;  // rows a block takes at a time
    from = blockIdx.y * per + warp;
    step = gridDim.y * per;
    for (int r0 = blockIdx.y * per; r0 < nrows; r0 += step) {
      if (per == 1) {
        Joined one[1];
        join_rows<1, 8>(a, first, last, first + warp, 8, r0, nrows, lane, one);
        part[warp][0][lane] = one[0];
      } else {
        Joined acc[kJoinRows];
        join_rows<kJoinRows, 2>(a, first, last, first + warp, 8, r0, nrows, lane, acc);
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i) part[warp][i][lane] = acc[i];
      }
      __syncthreads();
      if (warp < per && r0 + warp < nrows) {
        Joined x = part[0][warp][lane];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
          const Joined &y = part[i][warp][lane];
          join_one(x, y.m, y.l, y.o);
        }
        odd |= combine_store<T>(a, u, w.x, r0 + warp, lane, x);
      }
      __syncthreads();
    }
  }
  if (odd) mend_rows<T>(a, u, w.x, from, step, count, lane);  // (seldom)
}

template <class K>
cudaError_t core_go(K kernel, int bytes, const ChunkArgs &a, int ctas, cudaStream_t st) {
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(ctas), dim3(kThreads), bytes, st, a);
}

}  // namespace

cudaError_t launch_chunk_core(const ChunkArgs &a, bool q8, int rows, int ctas, cudaStream_t st) {
  if (rows == 4)
    return q8 ? core_go(chunk_rows_kernel<4, true>, sizeof(FewShared<4>), a, ctas, st)
              : core_go(chunk_rows_kernel<4, false>, sizeof(FewShared<4>), a, ctas, st);
  if (rows == 8)
    return q8 ? core_go(chunk_rows_kernel<8, true>, sizeof(FewShared<8>), a, ctas, st)
              : core_go(chunk_rows_kernel<8, false>, sizeof(FewShared<8>), a, ctas, st);
  return q8 ? core_go(chunk_core_kernel<true>, kTileSmem, a, ctas, st)
            : core_go(chunk_core_kernel<false>, kTileSmem, a, ctas, st);
}

cudaError_t launch_chunk_combine(int dtype, const ChunkArgs &a, int ctas, bool many,
                                 cudaStream_t st) {
  const int per = many ? 1 : kJoinRows;
  const dim3 grid(ctas, std::min(8, (a.slot_rows + per - 1) / per)), block(256);
  return dtype == KV_F32   ? launch_pdl(chunk_combine_kernel<float>, grid, block, 0, st, a)
         : dtype == KV_F16 ? launch_pdl(chunk_combine_kernel<__half>, grid, block, 0, st, a)
                           : launch_pdl(chunk_combine_kernel<__nv_bfloat16>, grid, block, 0, st, a);
}

}  // namespace kvs
