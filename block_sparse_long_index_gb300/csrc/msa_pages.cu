// The care of a paged cache: which pages a sequence holds, how many sequences
// hold a page, and the copies that forking and compacting need.
//
// A page is free when its count is 0; the call that needs pages takes the
// lowest free ones, in the order of its entries, so that a call's result does
// not depend on timing.  One CTA does what is ordered (checks, prefix sums, the
// search for free pages); tables and page contents are then written by a grid,
// its programmatic dependent, 16 KB of a page's pool a CTA at a time.
//
// Bound: the copies by HBM (a page read and written once), small calls by the
// two launches.  Measured: 8 sequences grown by a token and 56 forked from them
// (62 MB read and written, 1024 pages searched) 20 us for the two calls; 32
// sequences released and 2560 pages compacted, 643 MB read and written: 127 us,
// of which the copies take 93 (6.9 TB/s).
// What grows with the limits: the search for free pages goes through refs from
// page 0, 4096 at a time (64 entries of 8 pages: 9 us with 1024 pages, 13 us where
// the first 16384 of 32768 are held, 31 us where 100000 of 200000 are), compact's
// plan goes through all of them twice (25 us at 32768 pages, 119 us at 200000),
// and each entry is compared with those before it (1024 entries: 38 us, 4096:
// 271 us).
#include "msa_common.cuh"

namespace msa {

namespace {

constexpr int kThreads = 1024;
constexpr int kCopyThreads = 256;

// Scratch of a call: counters, the pages taken or moved, per-entry prefix sums, the page map.
struct PageScratch {
  int32_t* n_moves;  // pages to copy
  int32_t* from;     // [moves] page copied
  int32_t* to;       // [moves] into this one
  int32_t* len;      // [n] fork: the source's length when the call began
  int32_t* last;     // [n] fork: the new last page (-1: none)
  int32_t* map;      // [n_pages] compact: new id of each page
  int32_t* list;     // [n_pages] reserve: the free pages taken
};

// n > 0: reserve and fork with n entries; n = 0: compact.
size_t carve(const Pages& p, int n, char* base, PageScratch* w) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* r = base ? base + off : nullptr;
    off += align_up(bytes, 256);
    return r;
  };
  PageScratch s;
  const size_t moves = n > 0 ? (size_t)n : (size_t)p.n_pages;
  s.n_moves = (int32_t*)take(4);
  s.from = (int32_t*)take(moves * 4);
  s.to = (int32_t*)take(moves * 4);
  s.len = (int32_t*)take((size_t)n * 4);
  s.last = (int32_t*)take((size_t)n * 4);
  s.map = s.list = (int32_t*)take((size_t)p.n_pages * 4);  // one or the other
  if (w) *w = s;
  return off;
}

// Inclusive scan over the block; total = the block's sum.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // warp_sums of the scan before is no longer read
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    T w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[kThreads / 32 - 1];
  return v + (warp ? warp_sums[warp - 1] : T(0));
}

__device__ __forceinline__ int64_t pages_of(int64_t len, int page) { return (len + page - 1) / page; }

// Whether an earlier entry of the call names the same sequence (`names`: the entries in shared memory).
__device__ __forceinline__ bool named_before(const int* names, int i) {
  bool hit = false;
#pragma unroll 4
  for (int j = 0; j < i; ++j) hit |= names[j] == names[i];
  return hit;
}

// Lists the `need` lowest free pages in the scratch `list` (nothing else is changed, so a call that finds too few
// can give up).  Every thread takes part; returns how many were found.
__device__ __forceinline__ int list_free(const Pages& p, int need, int* warp_sums, int32_t* list) {
  int have = 0;
  for (int64_t b = 0; b < p.n_pages && have < need; b += kThreads * 4) {
    const int64_t i0 = b + threadIdx.x * 4;
    int32_t f[4];
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = i0 + j < p.n_pages ? p.refs[i0 + j] : 1;
#pragma unroll
    for (int j = 0; j < 4; ++j) n += f[j] == 0 ? 1 : 0;
    int total;
    int r = have + block_scan(n, warp_sums, total) - n;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (f[j] == 0) {
        if (r < need) list[r] = (int32_t)(i0 + j);
        ++r;
      }
    have += total;
  }
  __syncthreads();  // the list is whole
  return min(have, need);
}

// The entry whose run [pre[i], pre[i + 1]) holds r; pre has n + 1 values.
__device__ __forceinline__ int owner_of(const int* pre, int n, int r) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= r) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) pages_reserve_kernel(Pages p, const int32_t* __restrict__ seqs,
                                                                 const int32_t* __restrict__ new_len, int n, PageScratch w,
                                                                 DeviceStatus* st) {
  __shared__ int warp_sums[32];
  __shared__ int64_t need_sums[32];
  extern __shared__ int dyn[];
  int* names = dyn;          // [n]
  int* pre = dyn + n;        // [n + 1] pages needed before each entry (where they are as many as there are pages)
  const int tid = threadIdx.x;
  clear_errors(st);
  for (int i = tid; i < n; i += kThreads) names[i] = seqs[i];
  __syncthreads();
  int64_t carry = 0;
  int bad = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    int64_t need = 0;
    if (i < n) {
      const int32_t s = names[i], want = new_len[i];
      bool ok = s >= 0 && s < p.n_seqs && !named_before(names, i);
      if (ok) {
        const int32_t len = p.ctx[s];
        ok = len >= 0 && want >= len && (int64_t)want <= p.max_pages * p.page;
        if (ok) need = pages_of(want, p.page) - pages_of(len, p.page);
      }
      if (!ok) bad = 1;
    }
    int64_t total;
    const int64_t incl = block_scan(need, need_sums, total);
    if (i < n) pre[i] = (int)(carry + incl - need);
    carry += total;
  }
  if (tid == 0) pre[n] = (int)carry;
  if (__syncthreads_or(bad)) {
    if (tid == 0) raise_error(st, kErrBadIndex, 9u);
    return;
  }
  if (carry > p.n_pages || list_free(p, (int)carry, warp_sums, w.list) < (int)carry) {  // uniform
    if (tid == 0) raise_error(st, kErrNoPages, 10u);
    return;
  }
  for (int r = tid; r < (int)carry; r += kThreads) {
    const int i = owner_of(pre, n, r);
    const int32_t s = names[i], page = w.list[r];
    p.table[(int64_t)s * p.max_pages + pages_of(p.ctx[s], p.page) + (r - pre[i])] = page;
    p.refs[page] = 1;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) p.ctx[names[i]] = new_len[i];
}

// Checks the entries and gives each one whose source ends inside a page a new last page.
__global__ void __launch_bounds__(kThreads) pages_fork_plan_kernel(Pages p, const int32_t* __restrict__ src,
                                                                   const int32_t* __restrict__ dst, int n, PageScratch w,
                                                                   DeviceStatus* st) {
  __shared__ int warp_sums[32];
  extern __shared__ int dyn[];
  int* names = dyn;    // [n] dst
  int* pre = dyn + n;  // [n + 1]
  const int tid = threadIdx.x;
  griddep_launch_dependents();  // the copying grid waits for this one's end
  clear_errors(st);
  for (int i = tid; i < n; i += kThreads) names[i] = dst[i];
  __syncthreads();
  int carry = 0, bad = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    int need = 0;
    if (i < n) {
      const int32_t s = src[i], d = names[i];
      bool ok = s >= 0 && s < p.n_seqs && d >= 0 && d < p.n_seqs && !named_before(names, i);
      int32_t len = 0;
      if (ok) {
        len = p.ctx[s];
        ok = p.ctx[d] == 0 && len >= 0 && (int64_t)len <= p.max_pages * p.page;
        if (ok && len % p.page) {
          need = 1;
          const int32_t last = p.table[(int64_t)s * p.max_pages + len / p.page];
          ok = last >= 0 && (int64_t)last < p.n_pages;
          w.from[i] = last;
        }
      }
      if (!ok) bad = 1;
      w.last[i] = -1;
      w.len[i] = ok ? len : 0;
    }
    int total;
    const int incl = block_scan(need, warp_sums, total);
    if (i < n) pre[i] = carry + incl - need;
    carry += total;
  }
  if (tid == 0) pre[n] = carry;
  bad = __syncthreads_or(bad);
  const bool room = !bad && list_free(p, carry, warp_sums, w.to) == carry;
  if (!room) {
    if (tid == 0) {
      raise_error(st, bad ? kErrBadIndex : kErrNoPages, 11u);
      *w.n_moves = -1;  // nothing is forked
    }
    return;
  }
  for (int r = tid; r < carry; r += kThreads) {
    const int32_t page = w.to[r];
    w.last[owner_of(pre, n, r)] = page;
    p.refs[page] = 1;
  }
  if (tid == 0) *w.n_moves = n;  // entries without a new page are passed over by the copy (last < 0)
}

// page_bytes of every pool from page a to page b, by the threads of one CTA.
__device__ __forceinline__ void copy_piece(const PagePools& pools, int pool, int64_t a, int64_t b, size_t off, size_t bytes) {
  const uint4* s = reinterpret_cast<const uint4*>(pools.base[pool] + a * pools.page_bytes[pool] + off);
  uint4* d = reinterpret_cast<uint4*>(pools.base[pool] + b * pools.page_bytes[pool] + off);
  for (size_t i = threadIdx.x; i < bytes / 16; i += kCopyThreads) d[i] = ldg_stream_16(s + i);
}

constexpr size_t kPiece = 16384;  // bytes a CTA copies at a time

template <typename F>
__device__ __forceinline__ void copy_moves(const PagePools& pools, int64_t moves, F move) {
  size_t per = 0;
  for (int i = 0; i < pools.n; ++i) per += (pools.page_bytes[i] + kPiece - 1) / kPiece;
  const int64_t pieces = moves * (int64_t)per;
  for (int64_t x = blockIdx.x; x < pieces; x += gridDim.x) {
    size_t k = (size_t)(x % (int64_t)per);
    int pool = 0;
    for (;; ++pool) {
      const size_t m = (pools.page_bytes[pool] + kPiece - 1) / kPiece;
      if (k < m) break;
      k -= m;
    }
    int32_t a, b;
    if (!move(x / (int64_t)per, a, b)) continue;
    const size_t off = k * kPiece, left = pools.page_bytes[pool] - off;
    copy_piece(pools, pool, a, b, off, left < kPiece ? left : kPiece);
  }
}

__global__ void __launch_bounds__(kCopyThreads) pages_fork_kernel(Pages p, const int32_t* __restrict__ src,
                                                                  const int32_t* __restrict__ dst, int n, PageScratch w,
                                                                  PagePools pools, DeviceStatus* st) {
  griddep_wait();  // the plan
  if (*w.n_moves < 0) return;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int32_t s = src[i], d = dst[i];
    const int32_t len = w.len[i];  // (the source may itself be an empty one that this call fills)
    const int64_t full = len / p.page;
    const int32_t* from = p.table + (int64_t)s * p.max_pages;
    int32_t* to = p.table + (int64_t)d * p.max_pages;
    for (int64_t j = threadIdx.x; j < full; j += kCopyThreads) {
      const int32_t id = from[j];
      to[j] = id;
      if (id >= 0 && (int64_t)id < p.n_pages) atomicAdd(&p.refs[id], 1);
      else raise_error(st, kErrBadIndex, 12u);
    }
    if (threadIdx.x == 0) {
      if (w.last[i] >= 0) to[full] = w.last[i];
      p.ctx[d] = len;
    }
  }
  copy_moves(pools, n, [&](int64_t i, int32_t& a, int32_t& b) {
    a = w.from[i];
    b = w.last[i];
    return b >= 0;
  });
}

// One CTA per entry: an entry with a bad id, or whose sequence an earlier entry names, is passed over.
__global__ void __launch_bounds__(kCopyThreads) pages_free_kernel(Pages p, const int32_t* __restrict__ seqs, int n,
                                                                  DeviceStatus* st) {
  const int i = blockIdx.x, tid = threadIdx.x;
  const int32_t s = seqs[i];
  int skip = 0;
  for (int j = tid; j < i; j += kCopyThreads) skip |= seqs[j] == s;
  if (__syncthreads_or(skip)) return;
  const int32_t len = s >= 0 && s < p.n_seqs ? p.ctx[s] : -1;
  int bad = len < 0 || (int64_t)len > p.max_pages * p.page;
  int32_t* row = p.table + (int64_t)(bad ? 0 : s) * p.max_pages;
  const int64_t held = bad ? 0 : pages_of(len, p.page);
  for (int64_t j = tid; j < held; j += kCopyThreads) bad |= row[j] < 0 || (int64_t)row[j] >= p.n_pages;
  if (__syncthreads_or(bad)) {
    if (tid == 0) raise_error(st, kErrBadIndex, 13u);
    return;
  }
  for (int64_t j = tid; j < held; j += kCopyThreads) {
    const int32_t id = row[j];
    row[j] = -1;
    if (atomicSub(&p.refs[id], 1) <= 0) {  // the page was free already
      atomicAdd(&p.refs[id], 1);
      raise_error(st, kErrBadIndex, 14u);
    }
  }
  if (tid == 0) p.ctx[s] = 0;
}

// The r-th free page below n_live takes in the r-th held page at or above it.
__global__ void __launch_bounds__(kThreads) pages_compact_plan_kernel(Pages p, PageScratch w, int32_t* __restrict__ map,
                                                                      int32_t* __restrict__ n_live_out, DeviceStatus* st) {
  __shared__ int warp_sums[32];
  __shared__ int n_live_s;
  const int tid = threadIdx.x;
  griddep_launch_dependents();  // the copying grid waits for this one's end
  clear_errors(st);
  int live = 0;
  for (int64_t i = tid; i < p.n_pages; i += kThreads) live += p.refs[i] > 0 ? 1 : 0;
  int total;
  block_scan(live, warp_sums, total);
  if (tid == 0) n_live_s = total;
  __syncthreads();
  const int64_t n_live = n_live_s;
  int holes = 0, movers = 0;
  for (int64_t b = 0; b < p.n_pages; b += kThreads * 4) {
    const int64_t i0 = b + tid * 4;
    int32_t f[4];
    int nh = 0, nm = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + j;
      f[j] = i < p.n_pages ? p.refs[i] : 0;
      nh += i < n_live && f[j] <= 0;
      nm += i >= n_live && f[j] > 0;
    }
    int th, tm;
    int rh = holes + block_scan(nh, warp_sums, th) - nh;
    int rm = movers + block_scan(nm, warp_sums, tm) - nm;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + j;
      if (i >= p.n_pages) continue;
      if (i < n_live) {
        if (f[j] <= 0) w.to[rh++] = (int32_t)i;
        map[i] = f[j] > 0 ? (int32_t)i : -1;
      } else {
        if (f[j] > 0) w.from[rm++] = (int32_t)i;
        map[i] = -1;  // a moved page's place follows when every hole is known
      }
    }
    holes += th;
    movers += tm;
  }
  __syncthreads();
  for (int r = tid; r < movers; r += kThreads) {
    const int32_t a = w.from[r], b = w.to[r];
    map[a] = b;
    p.refs[b] = p.refs[a];
    p.refs[a] = 0;
  }
  if (tid == 0) {
    *w.n_moves = movers;
    if (n_live_out) *n_live_out = (int32_t)n_live;
  }
}

__global__ void __launch_bounds__(kCopyThreads) pages_compact_kernel(Pages p, PageScratch w, const int32_t* __restrict__ map,
                                                                     PagePools pools, DeviceStatus* st) {
  griddep_wait();  // the plan
  for (int s = blockIdx.x; s < p.n_seqs; s += gridDim.x) {
    const int32_t len = p.ctx[s];
    if (len < 0 || (int64_t)len > p.max_pages * p.page) {
      if (threadIdx.x == 0) raise_error(st, kErrBadIndex, 15u);
      continue;
    }
    int32_t* row = p.table + (int64_t)s * p.max_pages;
    const int64_t held = pages_of(len, p.page);
    for (int64_t j = threadIdx.x; j < held; j += kCopyThreads) {
      const int32_t id = row[j];
      const int32_t to = id >= 0 && (int64_t)id < p.n_pages ? map[id] : -1;
      if (to >= 0) row[j] = to;
      else raise_error(st, kErrBadIndex, 16u);
    }
  }
  copy_moves(pools, *w.n_moves, [&](int64_t r, int32_t& a, int32_t& b) {
    a = w.from[r];
    b = w.to[r];
    return true;
  });
}

unsigned copy_grid() { return (unsigned)(num_sms() * 8); }

// The copying grid as a programmatic dependent of the single CTA before it.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), unsigned grid, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, (P)args...);
}

}  // namespace

size_t pages_scratch_bytes(const Pages& p, int n) { return carve(p, n, nullptr, nullptr); }

cudaError_t launch_pages_reserve(const Pages& p, const int32_t* seqs, const int32_t* new_len, int n, void* scratch,
                                 DeviceStatus* st, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  PageScratch w;
  carve(p, n, (char*)scratch, &w);
  pages_reserve_kernel<<<1, kThreads, (size_t)(2 * n + 1) * 4, s>>>(p, seqs, new_len, n, w, st);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const Pages& p, const int32_t* src, const int32_t* dst, int n, const PagePools& pools,
                              void* scratch, DeviceStatus* st, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  PageScratch w;
  carve(p, n, (char*)scratch, &w);
  pages_fork_plan_kernel<<<1, kThreads, (size_t)(2 * n + 1) * 4, s>>>(p, src, dst, n, w, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent(pages_fork_kernel, copy_grid(), s, p, src, dst, n, w, pools, st);
}

cudaError_t launch_pages_free(const Pages& p, const int32_t* seqs, int n, DeviceStatus* st, cudaStream_t s) {
  if (n > 0) pages_free_kernel<<<(unsigned)n, kCopyThreads, 0, s>>>(p, seqs, n, st);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const Pages& p, const PagePools& pools, int32_t* page_map, int32_t* n_live, void* scratch,
                                 DeviceStatus* st, cudaStream_t s) {
  PageScratch w;
  carve(p, 0, (char*)scratch, &w);
  int32_t* map = page_map ? page_map : w.map;
  pages_compact_plan_kernel<<<1, kThreads, 0, s>>>(p, w, map, n_live, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent(pages_compact_kernel, copy_grid(), s, p, w, (const int32_t*)map, pools, st);
}

}  // namespace msa
