// Dense causal attention over packed prompts (msa_dense_prefill_varlen).
//
// Sequence s holds rows [cu[s], cu[s+1]) of q, k and v; row t of it sees the
// rows cu[s] .. t:  O[t,h] = sum_j softmax_j(scale q[t,h].k[j,g]) v[j,g].
// A work item is a run of positions of one sequence; the planning kernel lists
// them with the ones that see most keys first, so that the short ones fill the
// end of the launch.
//
// Bound: the tensor cores, 4 d FLOP for every visible (row, key, head) pair;
// operands are read once from HBM and again from L2.  Measured, against a
// library bf16 product's 1913.8 TFLOP/s on the same GPU (1709 when it runs for
// seconds):
//   one prompt of 32768, 64 heads on 8, d = 128: 11.6 to 11.8 ms, 1490 to 1510
//   TFLOP/s (0.78 to 0.79); 10.7 ms, 1640 TFLOP/s (0.86) for a call after a pause -
//   calls in a row reach the board's 1400 W, and the clock falls from 2.07 to 1.88 GHz;
//   8 prompts of 167 to 16000 rows, 32 heads on 8: 1.95 to 1.98 ms, 1450 TFLOP/s
//   (0.75 to 0.76);
//   5 prompts of 1 to 640 rows, 32 heads on 8: 20 us, where start and end count;
//   d = 64, whose products take half as long while the softmax does not: 32768
//   rows, 64 heads on 8, 10.0 ms, 877 TFLOP/s (0.46), 16 on 16, 2.56 ms (0.45).
#include <math.h>

#include "msa_sm100.cuh"

namespace msa {

namespace {

using namespace sm100;

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
  griddep_launch_dependents();  // the attention's CTAs may set up meanwhile; they wait for this grid's end
  clear_errors(st);
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

// ---------------------------------------------------------------- attention
// One CTA per SM, persistent.  A work item is two query tiles of 128 rows (row
// = position * gs + head: 128 / gs positions x gs heads of one group) over the
// same keys; items are taken in the planned order, every other round backwards,
// so that the CTAs' sums stay even.  Per 128-key tile and query tile:
//   S = Q K^T -> TMEM;  P = 2^(S scale' - m) as bf16 over S's columns;  O += P V
// with O in TMEM.  The two query tiles alternate: while one's softmax runs, the
// tensor cores work on the other's P V and next S.  The running maximum is
// lazy: O and the row sum are rescaled only when a row's maximum has grown by
// more than 2^8, so P stays below 256 (its bf16 rounding is relative, so the
// factor costs no precision) and the rescale of O in TMEM is rare.  P's bf16 is
// what the product takes; sums, maxima and O are fp32.
//
// What bounds a step: the softmax.  A query tile's softmax takes some 1500
// cycles of the SM (512 of them exponentials, the rest the latencies of S's
// read, the maxima's exchange and P's write), the two tiles' products 2048 in
// 3000 (1024 at d = 64: tensor pipe 36 % active).  Measured and slower at 32K: 8 softmax warps a tile on both at once
// 12.4 ms; a tile's S read while the other's P is written 12.6 ms; P handed over
// in two parts 14.5 ms; 64-key steps 12.9 ms; exponentials under the old maximum
// before the exchange, done again where it proves too low, 11.7 ms.
// Warpgroups: 0 to 3 the softmax, of query tile 0 and 1 in turn: warpgroup h has
// keys 32 h .. + 31 of every row, and the four threads of a row exchange their
// maxima through shared memory.  (A tile's softmax lies between its S and its
// P V, so what counts is how long one takes: with two warpgroups for each tile
// it took 1670 cycles of 64 exponentials a thread against 1024 cycles of
// products.)  4 the output (O / l, lse), 5 one warp each for the TMA loads, the
// MMA issue of query tile 0 and 1, and the guard.  (With both tiles' products
// on one warp, each wait of it, some 150 cycles for a phase long complete, left
// the tensor cores idle: 11.9 ms at 32K and 64 heads against 11.7.)
//
// The guard makes the masked places of V harmless, because a weight of 0 times
// a NaN or an infinity would not be 0 on the tensor cores: in the key tiles
// that not every row of the item sees whole, it clears the rows past the item's
// last position and, from its first position on, any value that is not finite;
// the epilogue then adds the latter to the rows that do see them.
constexpr int kRowsT = 128, kKeysT = 128;
constexpr int kThreadsA = 768;
constexpr int kWarpEpi = 16, kWarpLoad = 20, kWarpMma = 21, kWarpGuard = 23;
constexpr float kLazy = 8.0f;
constexpr int kPoisonSlots = 8;
constexpr int kOwnRounds = 4;  // rounds that a CTA may plan for itself

template <int D>
struct Layout {
  static constexpr int NC = D / 64;                  // 64-column chunks
  static constexpr int CHUNK = 128 * 128;            // bytes of one chunk of a 128-row tile
  static constexpr int TILE = NC * CHUNK;
  static constexpr int STAGES = D == 128 ? 4 : 8;    // K and V tiles in flight
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * TILE;
  static constexpr int OFF_ST = OFF_KV + STAGES * TILE;  // each row's sums (four parts): [2 tiles][128] x 16 bytes
  static constexpr int OFF_MM = OFF_ST + 2 * 128 * 16;   // each row's maximum: [2 tiles][128]
  static constexpr int OFF_MX = OFF_MM + 2 * 128 * 4;    // exchange of row maxima, two buffers: [2][128] x 16 bytes
  static constexpr int OFF_BAR = OFF_MX + 2 * 128 * 16;
  static constexpr int SMEM = 1024 + OFF_BAR + 512;
  static constexpr uint32_t TMEM_O = 256;            // S / P of tile q at 128 q, O of tile q (d columns) at 256 + 128 q
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void reg_fence16(uint32_t (&r)[16]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
// The four warps that hold a quarter of the rows meet (a named barrier each).
__device__ __forceinline__ void quarter_sync(int quarter) { asm volatile("bar.sync %0, 128;\n" ::"r"(1 + quarter) : "memory"); }
__device__ __forceinline__ bool finite_bf16x2(uint32_t w) {
  return (w & 0x7F80u) != 0x7F80u && (w & 0x7F800000u) != 0x7F800000u;
}

__device__ __forceinline__ uint4 lds_16(uint32_t at) {
  uint4 y;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w) : "r"(at));
  return y;
}
__device__ __forceinline__ void sts_16(uint32_t at, uint4 y) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w) : "memory");
}
__device__ __forceinline__ uint32_t drop_not_finite(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
  return w;
}
// Products and their completion by the one lane with `lead` set, predicated: with a branch around each batch the
// issuing warp lost some 90 cycles a batch (12.8 -> 11.9 ms at 32K, 64 heads).
__device__ __forceinline__ void mma_ss_if(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p, e;\nsetp.ne.b32 e, %5, 0;\nsetp.ne.b32 p, %4, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p, e;\nsetp.ne.b32 e, %5, 0;\nsetp.ne.b32 p, %4, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.b32 e, %1, 0;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar), "r"(lead)
      : "memory");
}
// The value that every lane of the warp has, in a uniform register.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// One item of the CTA's sequence of them, positions relative to the start of the sequence.
struct Item {
  int t0, len;   // first position, length of the sequence
  int row0, g;   // row of the sequence's first position, group
  int n[2];      // key tiles that query tile 0 and 1 see (0: no rows)
  __device__ __forceinline__ int n_max() const { return max(n[0], n[1]); }
};
struct Items {
  const int4* items;    // the planned list, or (own) this CTA's items by round
  bool own;
  int total, H_kv, PT;  // items x groups, groups, positions of a query tile
  __device__ __forceinline__ int index(int round) const {
    const int b = (int)blockIdx.x, n = (int)gridDim.x;
    return round * n + ((round & 1) ? n - 1 - b : b);
  }
  __device__ __forceinline__ bool get(int round, Item& it) const {
    const int i = index(round);
    if (i >= total) return false;
    load(round, it);
    return true;
  }
  __device__ __forceinline__ void load(int round, Item& it) const {
    const int i = index(round);
    const int4 x = items[own ? round : i / H_kv];
    it.g = i % H_kv;
    it.row0 = x.y;
    it.t0 = x.x - x.y;
    it.len = x.z - x.y;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int a = it.t0 + q * PT;
      it.n[q] = a < it.len ? (min(a + PT, it.len) - 1) / kKeysT + 1 : 0;
    }
  }
};

// The plan's list worked out by one warp for its CTA's few rounds, where S <= 32 (a lane a sequence) and the items give
// a CTA at most kOwnRounds: 5 prompts of 1 to 640 rows took 25.3 us with the planning kernel before it and 22.6 us so.
// (With more rounds it stops to matter: 8 prompts of 167 to 16000 rows, 28 rounds, 1961 us with the kernel, 1968 so.)
// Item i is of the largest depth d with more than i items at depth d or deeper.  Sequences of one depth go by their number.
__device__ __forceinline__ void plan_own(const int32_t* cu, int S, int64_t N, int P, int H_kv, int4* own, int* total,
                                         DeviceStatus* st) {
  const int lane = threadIdx.x & 31;
  const int32_t c0 = lane < S ? cu[lane] : 0, c1 = lane < S ? cu[lane + 1] : 0;
  const bool bad = lane < S && (c0 < 0 || c1 < c0 || (int64_t)c1 > N || (lane == 0 && c0 != 0));
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) {
      if (blockIdx.x == 0) raise_error(st, kErrBadIndex, 5u);
      *total = 0;
    }
    return;
  }
  const int n = (c1 - c0 + P - 1) / P, deepest = __reduce_max_sync(0xffffffffu, n);
  const int items = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) *total = items * H_kv;
  for (int r = 0; r < kOwnRounds; ++r) {
    const int at = r * (int)gridDim.x + ((r & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
    if (at >= items * H_kv) break;
    const int i = at / H_kv;
    int lo = 0, hi = deepest;  // the number of items at depth lo or deeper exceeds i, at hi it does not
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__reduce_add_sync(0xffffffffu, max(n - mid, 0)) > i) lo = mid; else hi = mid;
    }
    const int rank = i - __reduce_add_sync(0xffffffffu, max(n - lo - 1, 0));
    const unsigned who = __ballot_sync(0xffffffffu, n > lo);
    if (n > lo && __popc(who & ((1u << lane) - 1u)) == rank) own[r] = make_int4(c0 + lo * P, c0, c1, 0);
  }
}

template <int D, int GS>
__global__ void __launch_bounds__(kThreadsA, 1) dense_prefill_kernel(
    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
    const __grid_constant__ CUtensorMap tm_v, const uint16_t* __restrict__ v, const int32_t* __restrict__ cu, int own_S,
    int64_t N, int H_q, int H_kv, float scale_log2, DensePlanScratch w, uint16_t* __restrict__ out, float* __restrict__ lse, DeviceStatus* st) {
  using L = Layout<D>;
  constexpr int PT = kRowsT / GS;
  constexpr uint32_t IDESC_S = idesc_bf16_f32(kRowsT, kKeysT);
  constexpr uint32_t IDESC_PV = idesc_bf16_f32(kRowsT, D) | (1u << 16);  // V is MN-major
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(sm);
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int4 own_items[kOwnRounds];
  __shared__ int own_total;
  __shared__ int poison[kPoisonSlots];  // 1 + the round whose V tiles held values that are not finite
  const uint32_t bar = sb + L::OFF_BAR;
  auto kv_full = [&](int i) { return bar + 8u * i; };                    // TMA -> MMA, guard
  auto kv_empty = [&](int i) { return bar + 8u * (L::STAGES + i); };     // MMA (each tile's commit) -> TMA
  constexpr int B0 = 2 * L::STAGES;
  auto q_full = [&](int q) { return bar + 8u * (B0 + q); };              // TMA -> MMA
  auto q_empty = [&](int q) { return bar + 8u * (B0 + 2 + q); };         // MMA (commit) -> TMA
  auto s_full = [&](int q) { return bar + 8u * (B0 + 4 + q); };          // MMA (commit) -> softmax
  auto p_full = [&](int q) { return bar + 8u * (B0 + 6 + q); };          // softmax (16 warps) -> MMA
  auto pv_done = [&](int q) { return bar + 8u * (B0 + 8 + q); };         // MMA (commit) -> softmax
  auto o_full = [&](int q) { return bar + 8u * (B0 + 10 + q); };         // MMA (commit) -> output
  auto o_empty = [&](int q) { return bar + 8u * (B0 + 12 + q); };        // output (4 warps) -> MMA, softmax
  auto ml_full = [&](int q) { return bar + 8u * (B0 + 14 + q); };        // softmax (16 warps) -> output
  // V tiles alone, which sit in the odd stages; one a stage, so that the guard cannot be two phases ahead
  auto v_ok = [&](int i) { return bar + 8u * (B0 + 16 + i / 2); };       // guard -> MMA
  auto drain = [&](int q) { return bar + 8u * (B0 + 16 + L::STAGES / 2 + q); };
  static_assert(L::STAGES % 2 == 0 && 8 * (B0 + 18 + L::STAGES / 2) <= 512, "K and V alternate; barriers fit");
  float4* ml_s = reinterpret_cast<float4*>(sm + L::OFF_ST);
  float* mm_s = reinterpret_cast<float*>(sm + L::OFF_MM);
  float* mx_s = reinterpret_cast<float*>(sm + L::OFF_MX);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < L::STAGES; ++i) {
      mbar_init(kv_full(i), 1);
      mbar_init(kv_empty(i), 2);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(drain(q), 1);
      mbar_init(q_full(q), 1);
      mbar_init(q_empty(q), 1);
      mbar_init(s_full(q), 1);
      mbar_init(p_full(q), 16);
      mbar_init(pv_done(q), 1);
      mbar_init(o_full(q), 1);
      mbar_init(o_empty(q), 4);
      mbar_init(ml_full(q), 16);
    }
    for (int i = 1; i < L::STAGES; i += 2) mbar_init(v_ok(i), 1);
    fence_mbar_init();
    abort_flag = 0;
    for (int i = 0; i < kPoisonSlots; ++i) poison[i] = 0;
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tc_fence_before();
  }
  if (warp == kWarpLoad && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (own_S && warp == kWarpGuard) plan_own(cu, own_S, N, 2 * PT, H_kv, own_items, &own_total, st);
  __syncthreads();
  tc_fence_after();
  griddep_wait();  // the plan, where there is one
  const uint32_t tmem = tmem_slot;
  volatile int* abort = &abort_flag;
  Items items;
  items.own = own_S != 0;
  items.items = own_S ? own_items : w.items;
  items.total = own_S ? own_total : *w.n_items * H_kv;
  items.H_kv = H_kv;
  items.PT = PT;
  Item it;

  if (warp >= kWarpLoad) {
    if (warp == kWarpLoad) {
      // ------------------------------------------------------------ TMA
      if (lane == 0) {
        uint32_t kv = 0, qn[2] = {0, 0};
        bool ok = true;
        auto load_kv = [&](const CUtensorMap* map, int j) {
          const int s = (int)(kv % L::STAGES);
          if (!(ok = mbar_wait(kv_empty(s), ((kv / L::STAGES) & 1) ^ 1, abort, st, 0xD01))) return;
          mbar_arrive_expect_tx(kv_full(s), (uint32_t)L::TILE);
#pragma unroll
          for (int c = 0; c < L::NC; ++c)
            tma_load_3d(sb + L::OFF_KV + s * L::TILE + c * L::CHUNK, map, c * 64, it.g, it.row0 + j * kKeysT, kv_full(s));
          ++kv;
        };
        auto load_q = [&](int q) {
          if (!(ok = mbar_wait(q_empty(q), (qn[q] & 1) ^ 1, abort, st, 0xD02))) return;
          mbar_arrive_expect_tx(q_full(q), (uint32_t)L::TILE);
#pragma unroll
          for (int c = 0; c < L::NC; ++c)
            tma_load_3d(sb + L::OFF_Q + q * L::TILE + c * L::CHUNK, &tm_q, c * 64, it.g * GS, it.row0 + it.t0 + q * PT,
                        q_full(q));
          ++qn[q];
        };
        for (int r = 0; ok && items.get(r, it); ++r) {
          const int n = it.n_max();
          load_q(0);
          if (ok) load_kv(&tm_k, 0);
          if (ok && it.n[1]) load_q(1);
          if (ok) load_kv(&tm_v, 0);
          for (int j = 1; ok && j < n; ++j) {
            load_kv(&tm_k, j);
            if (ok) load_kv(&tm_v, j);
          }
        }
        if (!ok) {  // let the copies in flight land before the CTA ends
          for (uint32_t x = kv > (uint32_t)L::STAGES ? kv - L::STAGES : 0; x < kv; ++x)
            mbar_wait(kv_full((int)(x % L::STAGES)), (x / L::STAGES) & 1, nullptr, st, 0xDF1);
          for (int q = 0; q < 2; ++q)
            if (qn[q]) mbar_wait(q_full(q), (qn[q] - 1) & 1, nullptr, st, 0xDF2);
        }
      }
    } else if (warp < kWarpGuard) {
      // ------------------------------------------------------------ MMA issue: warp kWarpMma + q for query tile q
      // The whole warp runs the loops on warp-uniform values and one elected lane issues: descriptors then live in
      // uniform registers.  (Run by one lane alone, the register moves of each product cost more than the product.)
      // A wait that gives up is not looked at: the later ones return at once, and every address stays in bounds.
      const int q = (int)uniform((uint32_t)(warp - kWarpMma));
      const uint32_t ts = uniform(tmem) + q * 128, to = ts + L::TMEM_O, lead = elect_one();
      const int total = (int)uniform((uint32_t)items.total);
      uint32_t ks = 0, kph = 0;  // stage of the next K tile (its V tile is the one after) and the parity of its use
      uint32_t sp = 0, ip = 0;   // parities: softmax results, items of the query tile
      const uint64_t qd = umma_desc_kmajor(sb + L::OFF_Q + q * L::TILE, 128);
      auto product_s = [&](bool on, bool q_last) {
        mbar_wait(kv_full(ks), kph, abort, st, 0xD11);  // (a tile that is passed over too: the ring is walked in step)
        if (on) {
          tc_fence_after();
          // a descriptor's low bits are the address / 16: the steps along d are added to it
          const uint64_t kd = umma_desc_kmajor(sb + L::OFF_KV + ks * L::TILE, 128);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * L::CHUNK + (k & 3) * 32) / 16;
            mma_ss_if(lead, ts, qd + off, kd + off, IDESC_S, k > 0);
          }
          commit_if(lead, s_full(q));
          commit_if(lead & (uint32_t)q_last, q_empty(q));
        }
        commit_if(lead, kv_empty(ks));
      };
      for (int r = 0; items.index(r) < total; ++r) {
        items.load(r, it);
        const int n = (int)uniform((uint32_t)it.n_max()), nq = (int)uniform((uint32_t)it.n[q]);
        if (nq) mbar_wait(q_full(q), ip, abort, st, 0xD10);
        product_s(nq > 0, nq == 1);
        for (int j = 0; j < n; ++j) {
          const uint32_t vs = ks + 1, vph = kph;
          ks += 2;  // the K tile of j + 1
          if (ks == (uint32_t)L::STAGES) ks = 0, kph ^= 1u;
          mbar_wait(v_ok(vs), vph, abort, st, 0xD14);  // (V is there, and guarded)
          if (j < nq) {
            const uint64_t vd = umma_desc_mnmajor_sw128(sb + L::OFF_KV + vs * L::TILE, L::CHUNK);
            if (j == 0) mbar_wait(o_empty(q), ip ^ 1u, abort, st, 0xD15);
            mbar_wait(p_full(q), sp, abort, st, 0xD16);
            sp ^= 1u;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kKeysT / 16; ++k)  // keys 16 k ..: part k / 2, packed from column 32 part on
              mma_ts_if(lead, to, ts + 32 * (k >> 1) + 8 * (k & 1), vd + k * (16 * 128 / 16), IDESC_PV,
                        (j > 0 || k > 0) ? 1u : 0u);
            commit_if(lead, pv_done(q));
            commit_if(lead & (uint32_t)(j + 1 == nq), o_full(q));
          }
          commit_if(lead, kv_empty(vs));
          if (j + 1 < n) product_s(j + 1 < nq, j + 2 == nq);
        }
        ip ^= (uint32_t)(nq > 0);
      }
      if (*abort) {  // the products in flight end before TMEM is released
        commit_if(lead, drain(q));
        mbar_wait(drain(q), 0, nullptr, st, 0xDF3);
      }
    } else {
      // ------------------------------------------------------------ guard
      uint32_t kv = 0;
      bool ok = true;
      for (int r = 0; ok && items.get(r, it); ++r) {
        const int n = it.n_max(), jd = it.t0 / kKeysT;
        const int t_end = min(it.t0 + 2 * PT, it.len);  // past the item's last position
        for (int j = 0; j < n; ++j) {
          const uint32_t x = kv + 2 * j + 1;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(kv_full((int)(x % L::STAGES)), (x / L::STAGES) & 1, abort, st, 0xD20))))
            break;
          if (j < jd) {  // every row of the item sees the whole tile
            if (lane == 0) mbar_arrive(v_ok((int)(x % L::STAGES)));
            continue;
          }
          // lane: 16-byte piece lane % 8 of a chunk's row lane / 8; rows before the item's first position are seen by all
          const uint32_t va = sb + L::OFF_KV + (x % L::STAGES) * L::TILE + (lane & 7) * 16;
          const int rows = min(128, t_end - j * kKeysT);  // of the tile, up to the item's last position
          bool found = false;
          for (int r0 = (max(it.t0 - j * kKeysT, 0) & ~7) + (lane >> 3); r0 - (lane >> 3) < rows; r0 += 16) {
            uint4 y[4][L::NC];
            uint32_t most = 0u;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int c = 0; c < L::NC; ++c) y[u][c] = r0 + 4 * u < rows ? lds_16(va + c * L::CHUNK + (r0 + 4 * u) * 128) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int c = 0; c < L::NC; ++c)
                most = __vmaxu2(most, __vmaxu2(__vmaxu2(y[u][c].x & 0x7FFF7FFFu, y[u][c].y & 0x7FFF7FFFu),
                                               __vmaxu2(y[u][c].z & 0x7FFF7FFFu, y[u][c].w & 0x7FFF7FFFu)));
            if (finite_bf16x2(most)) continue;
            found = true;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int c = 0; c < L::NC; ++c)
                if (r0 + 4 * u < rows)
                  sts_16(va + c * L::CHUNK + (r0 + 4 * u) * 128, make_uint4(drop_not_finite(y[u][c].x), drop_not_finite(y[u][c].y),
                                                                        drop_not_finite(y[u][c].z), drop_not_finite(y[u][c].w)));
          }
#pragma unroll 4
          for (int row = max(rows, 0) + (lane >> 3); row < 128; row += 4)
#pragma unroll
            for (int c = 0; c < L::NC; ++c) sts_16(va + c * L::CHUNK + row * 128, make_uint4(0u, 0u, 0u, 0u));
          if (found) poison[r % kPoisonSlots] = r + 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(v_ok((int)(x % L::STAGES)));
        }
        kv += 2 * n;
      }
    }
  } else if (warp >= kWarpEpi) {
    // ------------------------------------------------------------ output: a thread per row
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const int pos = row / GS, hh = row % GS;
    uint32_t in[2] = {0, 0};
    bool ok = true;
    for (int r = 0; ok && items.get(r, it); ++r) {
#pragma unroll 1
      for (int q = 0; ok && q < 2; ++q) {
        if (it.n[q] == 0) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(ml_full(q), in[q] & 1, abort, st, 0xD30) &&
                                         mbar_wait(o_full(q), in[q] & 1, abort, st, 0xD31));
        if (!ok) break;
        ++in[q];
        tc_fence_after();
        const float4 ml = ml_s[q * 128 + row];
        const float m = mm_s[q * 128 + row], sum = (ml.x + ml.y) + (ml.z + ml.w);
        const int t = it.t0 + q * PT + pos;
        const bool live = t < it.len;
        const bool bad = poison[r % kPoisonSlots] == r + 1;
        // scores of -inf alone leave a sum of 0: out 0 (0 / 0 otherwise), lse -inf
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        const int64_t grow = (int64_t)it.row0 + t;
        const int h = it.g * GS + hh;
        uint4* orow = reinterpret_cast<uint4*>(out + (grow * H_q + h) * D);
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t x[16];
          tmem_ld_x16(tmem + ((uint32_t)(quarter * 32) << 16) + L::TMEM_O + q * 128 + c * 16, x);
          tmem_ld_wait();
          reg_fence16(x);
          if (bad && live)  // the values that the guard took out, for the rows that see them
            for (int j = it.t0 & ~7; j <= t; ++j) {
              const uint16_t* vr = v + (((int64_t)it.row0 + j) * H_kv + it.g) * D + c * 16;
              for (int e = 0; e < 16; ++e) {
                const uint32_t b = vr[e];
                if ((b & 0x7F80u) == 0x7F80u) {
                  const float add = __uint_as_float(b << 16);
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    if (i == e) x[i] = __float_as_uint(__uint_as_float(x[i]) + add);
                }
              }
            }
          if (live)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t y[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                y[i] = pack_bf16x2(__uint_as_float(x[8 * e + 2 * i]) * inv, __uint_as_float(x[8 * e + 2 * i + 1]) * inv);
              orow[c * 2 + e] = make_uint4(y[0], y[1], y[2], y[3]);
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_empty(q));
        if (live) lse[(int64_t)h * N + grow] = (m + lg2_approx(sum)) * 0.69314718055994530942f;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax: keys 32 part .. + 31 of both query tiles
    constexpr int PK = kKeysT / 4;
    const int part = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t scol0 = tmem + ((uint32_t)(quarter * 32) << 16) + part * PK;
    const uint32_t ocol0 = tmem + ((uint32_t)(quarter * 32) << 16) + L::TMEM_O + part * (D / 4);
    const float kInf = __int_as_float(0x7f800000);
    const uint64_t sc2 = f2_pack(scale_log2, scale_log2);
    uint32_t sn[2] = {0, 0}, in[2] = {0, 0}, ex = 0;  // S products and items of each tile so far; exchanges
    // (A wait that gave up is not looked at: the later ones return at once, and the warps of a quarter stay in step.)
    for (int r = 0; items.get(r, it); ++r) {
      const int n = it.n_max();
      const int t0 = min(it.t0 + row / GS, it.len - 1), t1 = min(it.t0 + PT + row / GS, it.len - 1);  // past it: the last row
      float m[2] = {-kInf, -kInf};
      uint64_t l2[2] = {0, 0};
      for (int j = 0; j < n; ++j) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (j >= it.n[q]) continue;
          mbar_wait(s_full(q), sn[q] & 1, abort, st, 0xD40);
          __syncwarp();
          tc_fence_after();
          uint32_t x[32];
          tmem_ld_x32(scol0 + q * 128, x);
          tmem_ld_wait();
          reg_fence32(x);
          const int lim = (q ? t1 : t0) - j * kKeysT - part * PK;  // last visible column
          if (__any_sync(0xffffffffu, lim < PK - 1)) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e > lim) x[e] = 0xff800000u;
          }
          float m4[4] = {-kInf, -kInf, -kInf, -kInf};
#pragma unroll
          for (int e = 0; e < 32; e += 2) m4[(e >> 1) & 3] = max3(m4[(e >> 1) & 3], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          // two buffers: who writes one again has met the other warps since they read it
          float* mx = mx_s + ((ex & 1) * 128 + row) * 4;
          ++ex;
          mx[part] = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
          quarter_sync(quarter);
          const float4 mo = *reinterpret_cast<const float4*>(mx);
          const float mt = fmaxf(max3(mo.x, mo.y, mo.z), mo.w) * scale_log2;
          const bool grow = mt > m[q] + kLazy;  // the threads of a row decide alike
          if (__any_sync(0xffffffffu, grow)) {
            const float alpha = !grow ? 1.f : ex2_approx(m[q] - mt);  // 2^-inf = 0 at the first tile
            if (grow) m[q] = mt;
            float a, b;
            f2_unpack(l2[q], a, b);
            l2[q] = f2_pack(a * alpha, b * alpha);
            if (j > 0) {  // O holds the products up to tile j - 1; this part's columns of it
              mbar_wait(pv_done(q), (sn[q] - 1) & 1, abort, st, 0xD41);
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 64; ++c) {
                uint32_t o[16];
                tmem_ld_x16(ocol0 + q * 128 + c * 16, o);
                tmem_ld_wait();
                reg_fence16(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st_x16(ocol0 + q * 128 + c * 16, o);
              }
            }
          }
          const float mz = m[q] == -kInf ? 0.f : m[q];  // scores of -inf alone weigh 0
          const uint64_t nm2 = f2_pack(-mz, -mz);
          uint32_t pk[16];
          uint64_t ls[2] = {l2[q], 0};
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float a0, a1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), sc2, nm2), a0, a1);
            a0 = ex2_approx(a0);
            a1 = ex2_approx(a1);
            ls[(e >> 1) & 1] = f2_add(ls[(e >> 1) & 1], f2_pack(a0, a1));
            pk[e >> 1] = pack_bf16x2(a0, a1);
          }
          l2[q] = f2_add(ls[0], ls[1]);
          tmem_st_x16(scol0 + q * 128, pk);  // keys of this part -> its first 16 columns, packed
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(q));
          ++sn[q];
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (it.n[q] == 0) continue;
        // the output warps have read the item before's (m, l) once they gave O back
        mbar_wait(o_empty(q), (in[q] & 1) ^ 1, abort, st, 0xD42);
        __syncwarp();
        ++in[q];
        float a, b;
        f2_unpack(l2[q], a, b);
        reinterpret_cast<float*>(ml_s + q * 128 + row)[part] = a + b;
        if (part == 0) mm_s[q * 128 + row] = m[q];
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_full(q));
      }
    }
  }

  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int GS>
cudaError_t launch_t(const void* q, const void* k, const void* v, const int32_t* cu, const DensePlan& p,
                     const DensePlanScratch& w, float scale, void* out, float* lse, DeviceStatus* st, cudaStream_t s) {
  using L = Layout<D>;
  alignas(64) unsigned char tq[128], tk[128], tv[128];
  const uint64_t row = (uint64_t)D * 2;
  // q [N][H_q][d] as boxes {64 dims, gs heads, 128 / gs positions}; k, v [N][H_kv][d] as {64, 1, 128 rows}
  if (!encode_tmap_3d(tq, q, D, (uint64_t)p.H_q, (uint64_t)p.N, row, (uint64_t)p.H_q * row, 64, GS, kRowsT / GS, 128) ||
      !encode_tmap_3d(tk, k, D, (uint64_t)p.H_kv, (uint64_t)p.N, row, (uint64_t)p.H_kv * row, 64, 1, kKeysT, 128) ||
      !encode_tmap_3d(tv, v, D, (uint64_t)p.H_kv, (uint64_t)p.N, row, (uint64_t)p.H_kv * row, 64, 1, kKeysT, 128))
    return cudaErrorInvalidValue;
  auto kern = dense_prefill_kernel<D, GS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t most = p.max_items * p.H_kv;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(most < num_sms() ? most : num_sms()));
  cfg.blockDim = dim3(kThreadsA);
  cfg.dynamicSmemBytes = L::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.own ? 0 : 1;  // (a CTA that plans for itself reads cu before it waits)
  return cudaLaunchKernelEx(&cfg, kern, *reinterpret_cast<const CUtensorMap*>(tq), *reinterpret_cast<const CUtensorMap*>(tk),
                            *reinterpret_cast<const CUtensorMap*>(tv), (const uint16_t*)v, cu, p.own ? p.S : 0, p.N, p.H_q,
                            p.H_kv, scale * 1.4426950408889634f, w, (uint16_t*)out, lse, st);
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
  p.P = 2 * kRowsT / (H_q / H_kv);
  // a sequence of n > 0 rows has ceil(n / P) <= n / P + 1 items
  p.max_items = N / p.P + (S < N ? S : N);
  p.own = S <= 32 && p.max_items * H_kv <= (int64_t)kOwnRounds * num_sms();
  return p;
}

size_t dense_scratch_bytes(const DensePlan& p) { return carve(p, nullptr, nullptr); }

cudaError_t launch_dense_prefill(const void* q, const void* k, const void* v, const int32_t* cu, const DensePlan& p,
                                 float scale, void* out, float* lse, void* scratch, DeviceStatus* st, cudaStream_t s) {
  DensePlanScratch w;
  carve(p, (char*)scratch, &w);
  if (!p.own) {
    dense_plan_kernel<<<1, kPlanThreads, 0, s>>>(cu, p.S, p.N, p.P, w, (int)depths_of(p.N, p.P), st);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  using Fn = cudaError_t (*)(const void*, const void*, const void*, const int32_t*, const DensePlan&, const DensePlanScratch&, float,
                             void*, float*, DeviceStatus*, cudaStream_t);
  static const Fn table[2][4] = {{launch_t<64, 1>, launch_t<64, 2>, launch_t<64, 4>, launch_t<64, 8>},
                                 {launch_t<128, 1>, launch_t<128, 2>, launch_t<128, 4>, launch_t<128, 8>}};
  const int gs = p.H_q / p.H_kv;
  return table[p.d == 128][gs == 1 ? 0 : gs == 2 ? 1 : gs == 4 ? 2 : 3](q, k, v, cu, p, w, scale, out, lse, st, s);
}

}  // namespace msa
