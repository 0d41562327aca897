// Dense causal attention over packed prompts (msa_dense_prefill_varlen).
//
// Sequence s holds rows [cu[s], cu[s+1]) of q, k and v; row t of it sees the
// rows cu[s] .. t:  O[t,h] = sum_j softmax_j(scale q[t,h].k[j,g]) v[j,g].
// A work item is a run of positions of one sequence; the planning kernel lists
// them with the ones that see most keys first, so that the short ones fill the
// end of the launch.
#include <math.h>

#include "msa_common.cuh"
#include "msa_tiles.cuh"

namespace msa {

namespace {

using namespace tiles;

constexpr int kPlanThreads = 1024;

// Inclusive scan over the block (kPlanThreads threads); `total` is the block's sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // warp_sums of the scan before is no longer read
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[kPlanThreads / 32 - 1];
  return v + (warp ? warp_sums[warp - 1] : 0);
}

// One CTA.  first[s] = number of items before sequence s; an item's depth is its index within its sequence,
// and items are listed by falling depth (the order among equal depths is free: items are independent).
__global__ void __launch_bounds__(kPlanThreads) dense_plan_kernel(const int32_t* __restrict__ cu, int S, int64_t N, int P,
                                                                  DensePlanScratch w, int depths, DeviceStatus* st) {
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x;
  int bad = 0;
  for (int s = tid; s <= S; s += kPlanThreads) {
    const int32_t c = cu[s];
    if (c < 0 || (int64_t)c > N || (s == 0 && c != 0) || (s > 0 && c < cu[s - 1])) bad = 1;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      raise_error(st, kErrBadIndex, 5u);
      *w.n_items = 0;
    }
    return;
  }
  for (int i = tid; i <= depths; i += kPlanThreads) w.depth[i] = 0;
  __syncthreads();
  int carry = 0;
  for (int s0 = 0; s0 < S; s0 += kPlanThreads) {
    const int s = s0 + tid;
    const int n = s < S ? (cu[s + 1] - cu[s] + P - 1) / P : 0;
    int total;
    const int incl = block_scan(n, warp_sums, total);
    if (s < S) {
      w.first[s] = carry + incl - n;
      if (n > 0) atomicAdd(&w.depth[n - 1], 1);  // the deepest item's depth
    }
    carry += total;
  }
  const int n_items = carry;
  if (tid == 0) {
    w.first[S] = n_items;
    *w.n_items = n_items;
  }
  __syncthreads();
  // from the deepest: sequences that reach depth i, and items deeper than i
  int reach = 0, deeper = 0;
  for (int top = depths - 1; top >= 0; top -= kPlanThreads) {
    const int i = top - tid;
    int total;
    const int r = reach + block_scan(i >= 0 ? w.depth[i] : 0, warp_sums, total);
    reach += total;
    const int incl = block_scan(i >= 0 ? r : 0, warp_sums, total);
    if (i >= 0) w.depth[i] = deeper + incl - r;  // where the items of depth i begin
    deeper += total;
  }
  __syncthreads();
  for (int f = tid; f < n_items; f += kPlanThreads) {
    int lo = 0, hi = S;  // the sequence with first[s] <= f < first[s + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (w.first[mid] <= f) lo = mid; else hi = mid;
    }
    const int i = f - w.first[lo];
    const int at = atomicAdd(&w.depth[i], 1);
    w.items[at] = make_int4(cu[lo] + i * P, cu[lo], cu[lo + 1], 0);
  }
}

constexpr int kRows = 64, kKeys = 64, kThreads = 128;

// One CTA per (item, group): 64 rows = 64 / gs positions x gs heads, row = position * gs + head; keys in tiles
// of 64 through shared memory, online softmax in registers.
template <int D>
__global__ void __launch_bounds__(kThreads) dense_prefill_kernel(const uint16_t* __restrict__ q,
                                                                 const uint16_t* __restrict__ kc,
                                                                 const uint16_t* __restrict__ vc, int64_t N, int H_q,
                                                                 int H_kv, float scale, DensePlanScratch w,
                                                                 uint16_t* __restrict__ out, float* __restrict__ lse) {
  extern __shared__ __align__(16) uint16_t sm[];
  const int item = blockIdx.x / H_kv, g = blockIdx.x % H_kv, gs = H_q / H_kv;
  if (item >= *w.n_items) return;
  const int4 it = w.items[item];
  const int64_t t0 = it.x, seq0 = it.y, seq1 = it.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint16_t* qs = sm;
  uint16_t* ks = sm + kRows * D;
  uint16_t* vs = ks + kKeys * D;
  const int64_t kv_row = (int64_t)H_kv * D;
  load_rows(qs, kRows, D, q, [&](int r) -> const uint16_t* {
    const int64_t t = t0 + r / gs;
    return t < seq1 ? q + (t * H_q + (int64_t)g * gs + r % gs) * D : nullptr;
  });
  cp_async_commit();
  const int64_t t_last = min(t0 + kRows / gs, seq1) - 1;
  const float sl2 = scale * 1.4426950408889634f;
  float o[D / 8][4], m[2], l[2];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  m[0] = m[1] = __int_as_float(0xff800000);
  l[0] = l[1] = 0.f;
  int64_t row_t[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) row_t[e] = t0 + (warp * 16 + (lane >> 2) + 8 * e) / gs;
  for (int64_t j0 = seq0; j0 <= t_last; j0 += kKeys) {
    __syncthreads();
    auto src = [&](const uint16_t* base) {
      return [=](int r) -> const uint16_t* { return j0 + r < seq1 ? base + (j0 + r) * kv_row + (int64_t)g * D : nullptr; };
    };
    load_rows(ks, kKeys, D, kc, src(kc));
    load_rows(vs, kKeys, D, vc, src(vc));
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
    float s[kKeys / 8][4];
#pragma unroll
    for (int i = 0; i < kKeys / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D; kk += 16) {
      uint32_t a[4];
      lds_a(a, smem_u32(qs), warp * 16, kk, D);
#pragma unroll
      for (int n = 0; n < kKeys; n += 16) {
        uint32_t b[4];
        lds_b_nk(b, smem_u32(ks), n, kk, D);
        mma2(s[n / 8], s[n / 8 + 1], a, b);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float mx = m[e];
#pragma unroll
      for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int64_t j = j0 + n * 8 + 2 * (lane & 3) + c;
          float& x = s[n][2 * e + c];
          x = j <= row_t[e] ? x * sl2 : __int_as_float(0xff800000);
          mx = fmaxf(mx, x);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float ms = mx == __int_as_float(0xff800000) ? 0.f : mx;
      const float alpha = exp2f(m[e] - ms);
      m[e] = mx;
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float& x = s[n][2 * e + c];
          x = exp2f(x - ms);
          sum += x;
        }
      l[e] = l[e] * alpha + sum;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][2 * e] *= alpha;
        o[i][2 * e + 1] *= alpha;
      }
    }
#pragma unroll
    for (int kk = 0; kk < kKeys; kk += 16) {
      uint32_t a[4];
      c_to_a(a, s[kk / 8], s[kk / 8 + 1]);
#pragma unroll
      for (int n = 0; n < D; n += 16) {
        uint32_t b[4];
        lds_b_kn(b, smem_u32(vs), kk, n, D);
        mma2(o[n / 8], o[n / 8 + 1], a, b);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float L = l[e];
    L += __shfl_xor_sync(0xffffffffu, L, 1);
    L += __shfl_xor_sync(0xffffffffu, L, 2);
    const int h = g * gs + (warp * 16 + (lane >> 2) + 8 * e) % gs;
    if (row_t[e] >= seq1) continue;
    const float inv = 1.f / L;
    uint32_t* orow = reinterpret_cast<uint32_t*>(out + (row_t[e] * H_q + h) * D);
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      orow[i * 4 + (lane & 3)] = pack_bf16x2(o[i][2 * e] * inv, o[i][2 * e + 1] * inv);
    if ((lane & 3) == 0) lse[(int64_t)h * N + row_t[e]] = (m[e] + log2f(L)) * 0.69314718055994530942f;
  }
}

int64_t depths_of(int64_t N, int P) { return ceil_div(N, P); }

size_t carve(const DensePlan& p, char* base, DensePlanScratch* w) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* r = base ? base + off : nullptr;
    off += align_up(bytes, 256);
    return r;
  };
  DensePlanScratch s;
  s.n_items = (int*)take(4);
  s.first = (int*)take((size_t)(p.S + 1) * 4);
  s.depth = (int*)take((size_t)(depths_of(p.N, p.P) + 1) * 4);
  s.items = (int4*)take((size_t)p.max_items * sizeof(int4));
  if (w) *w = s;
  return off;
}

}  // namespace

DensePlan dense_plan(int64_t N, int S, int H_q, int H_kv, int d) {
  DensePlan p;
  p.N = N;
  p.S = S;
  p.H_q = H_q;
  p.H_kv = H_kv;
  p.d = d;
  p.P = kRows / (H_q / H_kv);
  // a sequence of n > 0 rows has ceil(n / P) <= n / P + 1 items
  p.max_items = N / p.P + (S < N ? S : N);
  return p;
}

size_t dense_scratch_bytes(const DensePlan& p) { return carve(p, nullptr, nullptr); }

cudaError_t launch_dense_prefill(const void* q, const void* k, const void* v, const int32_t* cu, const DensePlan& p,
                                 float scale, void* out, float* lse, void* scratch, DeviceStatus* st, cudaStream_t s) {
  DensePlanScratch w;
  carve(p, (char*)scratch, &w);
  dense_plan_kernel<<<1, kPlanThreads, 0, s>>>(cu, p.S, p.N, p.P, w, (int)depths_of(p.N, p.P), st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const size_t smem = (size_t)(kRows + 2 * kKeys) * p.d * 2;
  auto kern = p.d == 64 ? dense_prefill_kernel<64> : dense_prefill_kernel<128>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(p.max_items * p.H_kv), kThreads, smem, s>>>((const uint16_t*)q, (const uint16_t*)k, (const uint16_t*)v,
                                                                p.N, p.H_q, p.H_kv, scale, w, (uint16_t*)out, lse);
  return cudaGetLastError();
}

}  // namespace msa
