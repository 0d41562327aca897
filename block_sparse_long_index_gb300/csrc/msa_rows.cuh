// Packed rows of new tokens and where a paged cache keeps them: looked up by the calls that store, load and append.
#pragma once

#include "msa_common.cuh"

namespace msa {

constexpr int kRowThreads = 256;

// Where packed row i, of one of the sequences, goes: the pool row of its token, or -1 (bad: flagged).
struct RowMap {
  const int32_t* cu;    // [S + 1]
  const int32_t* pos0;  // [S] token position of each sequence's first row
  const int32_t* table;
  int64_t max_pages, n_pages;
  int S, page;

  // (t_out: the row's token position, where there is a place for it)
  __device__ __forceinline__ int64_t row(int64_t i, DeviceStatus* st, int32_t* t_out = nullptr) const {
    int lo = 0, hi = S;  // a sequence with cu[lo] <= i < cu[lo + 1] (a search by halves ends whatever cu holds)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= i) lo = mid; else hi = mid;
    }
    const int64_t t = (int64_t)pos0[lo] + (i - cu[lo]);
    if (i < cu[lo] || i >= cu[lo + 1] || pos0[lo] < 0 || t >= max_pages * page) {
      raise_error(st, kErrBadIndex, 6u);
      return -1;
    }
    const int64_t lp = t / page;
    const int32_t pp = table[(int64_t)lo * max_pages + lp];
    if (pp < 0 || (int64_t)pp >= n_pages) {
      raise_error(st, kErrBadIndex, 7u);
      return -1;
    }
    if (t_out) *t_out = (int32_t)t;
    return (int64_t)pp * page + (t - lp * page);
  }
};

inline RowMap row_map(const int32_t* cu, int S, const int32_t* pos0, const int32_t* table, int64_t max_pages, int64_t n_pages,
                      int page) {
  RowMap m;
  m.cu = cu;
  m.pos0 = pos0;
  m.table = table;
  m.max_pages = max_pages;
  m.n_pages = n_pages;
  m.S = S;
  m.page = page;
  return m;
}

// The pool rows of the CTA's `n` packed rows from i0 on (and their token positions, where `pos` is given); `none` for
// those of no sequence.
// A call of at most kRowThreads rows has its status written by CTA 0 alone, which looks up all of them (the other CTAs
// report nothing): the error word then needs no clearing before the kernel, a launch of its own (48 tokens in and out
// 12.4 -> 10.2 us on the GPU).
__device__ __forceinline__ void look_up(const RowMap& map, int64_t N, int64_t i0, int n, int64_t none, int64_t* rows,
                                        DeviceStatus* st, int32_t* pos = nullptr) {
  __shared__ unsigned int est[2];
  const int64_t in0 = map.cu[0], in1 = min((int64_t)map.cu[map.S], N);
  auto row = [&](int64_t i, DeviceStatus* s, int32_t* p) { return i >= in0 && i < in1 ? map.row(i, s, p) : none; };
  if (!kv4_rows_report(N) || blockIdx.x) {
    for (int t = threadIdx.x; t < n; t += kRowThreads) rows[t] = row(i0 + t, kv4_rows_report(N) ? nullptr : st, pos ? pos + t : nullptr);
    __syncthreads();
    return;
  }
  DeviceStatus* own = reinterpret_cast<DeviceStatus*>(est);  // (an error touches its first two words)
  if (threadIdx.x == 0) est[0] = est[1] = 0u;
  __syncthreads();
  const int64_t r = row(threadIdx.x, own, pos && (int)threadIdx.x < n ? pos + threadIdx.x : nullptr);
  if ((int)threadIdx.x < n) rows[threadIdx.x] = r;
  __syncthreads();
  if (threadIdx.x == 0) {
    st->flags = own->flags;
    st->first_code = own->first_code;
  }
}

}  // namespace msa
