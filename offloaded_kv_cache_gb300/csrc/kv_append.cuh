// kv_append.cuh -- what the chunk appends share: a sequence's rows and pages, and the
// lengths of an append in place.  A is a kernel's argument block: q_start, bt, ctx,
// ctx_out, status, nphys, ps, maxP, total_q, max_q_len.
#pragma once

#include "kv_internal.cuh"

namespace kvs {

// A sequence's chunk: rows [q0, q0 + n), stored from position len on; n < 0
// when the sequence is skipped.
struct RowSpan {
  int q0, n, len;
};
template <class A> __device__ __forceinline__ RowSpan append_span(const A &a, int b) {
  const int q0 = a.q_start[b], q1 = a.q_start[b + 1], len = a.ctx[b];
  const long long cap = (long long)a.maxP * a.ps;
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.total_q && q1 - q0 <= a.max_q_len && len >= 0 &&
                  len + (long long)(q1 - q0) <= cap;
  return RowSpan{q0, ok ? q1 - q0 : -1, len};
}
// Whether every page the chunk touches is in range (the whole block asks).
template <class A> __device__ __forceinline__ bool pages_ok(const A &a, int b, const RowSpan &r) {
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

// lengths of a chunk append in place, after every block has read them
template <class A> __global__ void __launch_bounds__(256) advance_kernel(const A a) {
  pdl_wait();
  const int b = blockIdx.x;
  const RowSpan r = append_span(a, b);
  const bool ok = r.n >= 0 && pages_ok(a, b, r);
  __syncthreads();
  if (threadIdx.x == 0 && ok) a.ctx_out[b] = r.len + r.n;
}

}  // namespace kvs
