// Attention of a tree of drafted tokens over a paged cache (msa_tree_decode_paged, msa_tree_decode_paged_kv4).
//
// Node i of sequence b sees the context, tokens 0 .. ctx - 1 of the cache, and of the drafts, tokens ctx + j, those
// with j = i or above it in the tree:  O[b,i,h] = sum_j softmax_j(scale q[b,i,h].k[j,g]) v[j,g].
//
// The two parts are worked out apart, as partial softmaxes (O, maximum, sum).  The context needs no mask: all rows of a
// (sequence, K/V head) see all of it, T gs rows that share every key, a matrix product.  A node's own branch is a
// handful of keys that differ from row to row, at most 64 in all: the kernel that joins the partials does it.
//
// The context: all sequences' 128-token tiles are one list, whatever the lengths are; a CTA has one unit (K/V head, and
// group of rows where they are many) and an equal run of the list.  The CTAs of all units take the same runs at the same
// time: the heads of a token lie side by side in memory, and 64 bytes here and there (a 4-bit head row) would keep HBM to
// a fifth of its rate.  tree_context_kernel does a tile by tcgen05, S = Q K^T and O += P V
// with 128 query rows, Q and K, V in shared memory, S / P and O in TMEM.  Two streams of it alternate, so that one's
// softmax runs under the other's products:
//   up to 128 rows, and over a 4-bit cache always: one query tile, whose even and odd key tiles are the streams (their O
//   are merged at the run's end);
//   more rows over bf16 pages: two query tiles over the same keys.  (4-bit pages are expanded again for each 128 rows: a
//   tile's softmax takes as long, and the room of the second query tile holds the codes in flight.)
// Rows of a tile past the last one are computed on by the tensor cores alone; warps without a row rest.
// P is rounded to bf16 for the product with V, whose operands have one type (V's is bf16, or exact in it); scores, sums and O
// stay fp32.
// Over a 4-bit cache up to 32 rows of up to 8 K/V heads have a kernel of their own (msa_tree_few.cu).
//
// Measured, with the join: bf16 pages, 128 rows, 4 sequences of 262144 tokens: 636 us, HBM's rate (a tile takes 1955
// cycles where the caches stay in L2, 2825 from HBM); 256 rows, 16 sequences of 1200 to 12000 tokens: 128 us, 0.51 of HBM
// (101 us the context, whose two query tiles' softmax takes 3150 cycles a tile).  4-bit pages, 128 rows, 4 of 2^20 tokens:
// 2534 us, 0.45 of the tensor cores' and 0.27 of HBM's rate: a tile is 6900 warp instructions, issue slots 58 % and ALU
// 45 % busy (2950 cycles).  Tried there and no faster: expanding warps moved away from the schedulers of live rows, K's
// stage handed over before V's, two tiles of codes in registers (spills, which cost a trip to L2 each beside 227 KB of
// shared memory: 7453 us), waits with a suspend hint.
#include <math.h>

#include "msa_kv4.cuh"
#include "msa_sm100.cuh"
#include "msa_tree.cuh"

namespace msa {

namespace {

using namespace sm100;
using namespace kv4;

constexpr int kRowsT = 128;
constexpr int kMaxT = 64;  // nodes of a tree: a 64-bit mask
constexpr int kWarpMma = 16, kWarpLoad = 18, kWarpGuard = 19, kWarpExpand = 20;
constexpr int kUnitRows = 16;                   // tokens of a tile that an expanding warp takes
constexpr int kUnits = kKeysT / kUnitRows;      // warps that expand 4-bit codes
__host__ __device__ constexpr int ctx_threads(bool kv4) { return 32 * (kv4 ? kWarpExpand + kUnits : kWarpExpand); }
constexpr int kJoinThreads = 128, kJoinWarps = kJoinThreads / 32;
constexpr int kMaxRounds = 4;
constexpr float kLazy = 8.0f;  // log2 units a row maximum may grow before O is rescaled

// What a CTA begins a round with: its unit and its group's run of the tile list.
struct Round {
  int seq, off, left;  // tile `off` of sequence `seq`, so many tiles
  int unit, group;
};
// The tiles of a CTA, round by round and segment by segment: tiles [t0, t1) of one sequence for the round's unit.
struct Run {
  int round, rounds;
  int left, off;  // tiles not given out yet; the next one's index in sequence `seq`
  int seq, unit, group;
  int len, t0, t1;  // of the segment: context length, tiles
  __device__ __forceinline__ bool next(const TreeShape& sh, const Round* start) {
    while (left <= 0) {
      if (++round >= rounds) return false;
      const Round r = start[round];
      seq = r.seq, off = r.off, left = r.left, unit = r.unit, group = r.group;
    }
    int n;
    while (off >= (n = sh.tiles(seq))) {  // (ends: the runs add up to the sum over all sequences)
      off = 0;
      ++seq;
    }
    t0 = off;
    t1 = min(t0 + left, n);
    int t;
    sh.lengths(seq, len, t);
    left -= t1 - t0;
    off = t1;
    return true;
  }
};

__device__ __forceinline__ int64_t run_quota(int64_t total, int groups) { return total ? (total + groups - 1) / groups : 1; }

template <int D>
struct Layout {
  static constexpr int NC = D / 64;                // 64-channel chunks
  static constexpr int CHUNK = 128 * 128;          // bytes of a chunk of 128 rows
  static constexpr int TILE = NC * CHUNK;
  static constexpr int STAGES = D == 128 ? 4 : 8;  // K and V tiles in flight
  static constexpr uint32_t TMEM_O = 256;          // S / P of stream q at 128 q, O of stream q at 256 + 128 q
  // places in shared memory, with one or two query tiles
  __host__ __device__ static constexpr int kv_at(bool two) { return (two ? 2 : 1) * TILE; }
  __host__ __device__ static constexpr int misc_at(bool two) { return kv_at(two) + STAGES * TILE; }
  static constexpr int SUMS = 0, MAXIMA = 2 * 128 * 16, BARS = MAXIMA + 2 * 128 * 16, MISC = BARS + 512;
  // 4-bit pages: a tile's codes of K and of V, then their scales; and the tiles of them in flight
  static constexpr int CODES = kKeysT * D / 2, SCALES = kKeysT * kGroups, RAW = 2 * (CODES + SCALES), DEPTH = D == 128 ? 3 : 4;
  __host__ __device__ static constexpr int raw_at(bool two) { return (misc_at(two) + MISC + 1023) / 1024 * 1024; }
  __host__ __device__ static constexpr int smem(bool two, bool kv4) {
    return 1024 + (kv4 ? raw_at(two) + DEPTH * RAW : misc_at(two) + MISC);
  }
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, int32_t w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
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
__device__ __forceinline__ uint4 lds_16(uint32_t at) {
  uint4 y;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w) : "r"(at));
  return y;
}
__device__ __forceinline__ void sts_16(uint32_t at, uint4 y) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w) : "memory");
}
__device__ __forceinline__ uint32_t lds_2(uint32_t at) {
  uint16_t y;
  asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(y) : "r"(at));
  return y;
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on `bar` once this thread's cp.async so far have landed (one of the arrivals that the barrier expects).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}
// Products and their completion by the one lane with `lead` set, predicated.
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
// Registers a thread, for all four warps of a warpgroup.
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }
// The value that every lane of the warp has, in a uniform register.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// Half a row's codes as bf16 times 2^-18, word w at `to` ^ 16 w; zeros where it is not context.
template <int HW>
__device__ __forceinline__ void expand_half(const uint4 (&c)[HW], uint32_t scales, bool on, uint32_t to) {
  if (!on) {
#pragma unroll
    for (int w = 0; w < 4 * HW; ++w) sts_16(to ^ (w << 4), make_uint4(0u, 0u, 0u, 0u));
    return;
  }
  SubScale sc[2];  // its two groups
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const uint32_t b = scales >> (8 * x) & 0xFFu;
    sc[x] = sub_scale(b == kScaleNaN ? 0x7FFF7FFFu : b * 0x00100010u + kSubScaleBias * 0x00010001u);
  }
#pragma unroll
  for (int y = 0; y < HW; ++y) {
    const uint32_t cw[4] = {c[y].x, c[y].y, c[y].z, c[y].w};
#pragma unroll
    for (int x = 0; x < 4; ++x) sts_16(to ^ ((4 * y + x) << 4), expand8_sub(cw[x], sc[(4 * y + x) / (2 * HW)]));
  }
}

// The CTA's rounds.  Every thread takes part.  CTA 0 writes starts.
template <int THREADS>
__device__ __forceinline__ void find_rounds(const TreeShape& sh, int64_t* starts, int64_t* warp_sums, Round* start) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = THREADS / 32;
  const int per = (sh.B + THREADS - 1) / THREADS, b0 = min(tid * per, sh.B), b1 = min(b0 + per, sh.B);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += sh.tiles(b);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int64_t total = 0, off = 0;
  for (int w = 0; w < nw; ++w) {
    const int64_t x = warp_sums[w];
    if (w < warp) off += x;
    total += x;
  }
  const int64_t quota = run_quota(total, sh.groups);
  const int units = sh.H_kv * sh.RG;
  if (tid < sh.rounds) {
    const int item = blockIdx.x + tid * gridDim.x;
    Round r;
    r.group = item / units;
    r.unit = item % units;
    r.seq = r.off = 0;
    r.left = r.group < sh.groups ? (int)max(min(total - r.group * quota, quota), (int64_t)0) : 0;
    start[tid] = r;
  }
  __syncthreads();
  const int64_t first = off + incl - mine;
  for (int i = 0; i < sh.rounds; ++i) {
    const int64_t at = (blockIdx.x + i * gridDim.x) / units * quota;
    if (start[i].left <= 0 || at < first || at >= first + mine) continue;
    int64_t x = first;
    for (int b = b0; b < b1; ++b) {
      const int n = sh.tiles(b);
      if (at < x + n) {
        start[i].seq = b;
        start[i].off = (int)(at - x);
        break;
      }
      x += n;
    }
  }
  if (blockIdx.x == 0) {
    int64_t x = first;
    for (int b = b0; b < b1; ++b) {
      starts[b] = x;
      x += sh.tiles(b);
    }
    if (tid == 0) starts[sh.B] = quota;
  }
  __syncthreads();
}

template <int D, bool KV4>
__global__ void __launch_bounds__(ctx_threads(KV4), 1) tree_context_kernel(
    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    TreeShape sh, CacheMap map, Kv4Pool pool, int box_rows, float scale_log2, TreeScratch w, DeviceStatus* status) {
  using L = Layout<D>;
  constexpr uint32_t IDESC_S = idesc_bf16_f32(kRowsT, kKeysT);
  constexpr uint32_t IDESC_PV = idesc_bf16_f32(kRowsT, D) | (1u << 16);  // V is MN-major
  extern __shared__ uint8_t smraw[];
  const uint32_t sb = (smem_u32(smraw) + 1023u) & ~1023u;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ unsigned int est[2];
  __shared__ int64_t warp_sums[ctx_threads(KV4) / 32];
  __shared__ Round start[kMaxRounds];
  __shared__ Run runs_s[kWarpMma];
  DeviceStatus* st = reinterpret_cast<DeviceStatus*>(est);  // the CTA's own (an error touches its first two words)
  const int R = sh.T * sh.gs;
  const bool two = !KV4 && R > kRowsT;  // two query tiles a unit
  const uint32_t sm_kv = sb + L::kv_at(two), sm_misc = sb + L::misc_at(two), bar = sm_misc + L::BARS;
  auto kv_full = [&](int i) { return bar + 8u * i; };
  auto kv_empty = [&](int i) { return bar + 8u * (L::STAGES + i); };  // both MMA warps
  constexpr int B0 = 2 * L::STAGES;
  const uint32_t q_full = bar + 8u * B0, q_empty = bar + 8u * (B0 + 1);
  auto s_full = [&](int q) { return bar + 8u * (B0 + 2 + q); };   // MMA -> softmax
  auto p_full = [&](int q) { return bar + 8u * (B0 + 4 + q); };   // softmax -> MMA
  auto pv_done = [&](int q) { return bar + 8u * (B0 + 6 + q); };  // MMA -> softmax
  auto o_full = [&](int q) { return bar + 8u * (B0 + 8 + q); };   // MMA -> softmax, at the segment's end
  auto o_empty = [&](int q) { return bar + 8u * (B0 + 10 + q); }; // softmax -> MMA
  auto drain = [&](int q) { return bar + 8u * (B0 + 12 + q); };
  // TMA -> guard, for V tiles (odd stages) that end inside the tile: the guard then fills kv_full.  A barrier of their
  // own, so that the guard, who passes over all other tiles, sees every phase of it.
  auto v_part = [&](int i) { return bar + 8u * (B0 + 14 + i / 2); };
  constexpr int B1 = B0 + 14 + L::STAGES / 2;
  auto raw_full = [&](int i) { return bar + 8u * (B1 + i); };               // 4-bit codes: TMA and cp.async -> expanding warps
  auto raw_empty = [&](int i) { return bar + 8u * (B1 + L::DEPTH + i); };   // expanding warps -> loads
  static_assert(8 * (B1 + 2 * L::DEPTH) <= 512, "barriers fit");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();
  // quarters (32 rows) that some tile of a stream uses
  const int most[2] = {min(R, kRowsT), two ? min(sh.RG > 1 ? kRowsT : R - kRowsT, kRowsT) : min(R, kRowsT)};
  const int live_q[2] = {(most[0] + 31) / 32, (most[1] + 31) / 32};
  if (tid == 0) {
    for (int i = 0; i < L::STAGES; ++i) {
      mbar_init(kv_full(i), KV4 ? kUnits : 1);
      mbar_init(kv_empty(i), 2);
    }
    for (int i = 1; i < L::STAGES; i += 2) mbar_init(v_part(i), 1);
    for (int i = 0; i < L::DEPTH; ++i) {
      mbar_init(raw_full(i), 33);  // TMA's bytes, every lane's scales
      mbar_init(raw_empty(i), kUnits);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      mbar_init(s_full(q), 1);
      mbar_init(p_full(q), 4 * live_q[q]);
      mbar_init(pv_done(q), 1);
      mbar_init(o_full(q), 1);
      mbar_init(o_empty(q), 4 * live_q[q]);
      mbar_init(drain(q), 1);
    }
    fence_mbar_init();
    abort_flag = 0;
    est[0] = est[1] = 0u;
    if (blockIdx.x == 0) {  // the joining kernel reports into it
      status->flags = 0u;
      status->first_code = 0u;
    }
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
  find_rounds<ctx_threads(KV4)>(sh, w.starts, warp_sums, start);
  Run run;
  run.round = -1;
  run.rounds = sh.rounds;
  run.left = 0;
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  volatile int* abort = &abort_flag;
  // rows of query tile q of a unit, and whether stream q takes tile j of the segment
  auto rows_of = [&](int unit, int q) { return min(kRowsT, max(0, R - (unit % sh.RG) * (KV4 ? kRowsT : 2 * kRowsT) - (two ? q * kRowsT : 0))); };

  // 896 threads start with 72 registers each, 64512 in all; 512 x 80 + 384 x 56 = 62464
  if (KV4 && warp >= kWarpMma) regs_dec<56>();
  if (warp >= kWarpLoad) {
    if (warp == kWarpLoad) {
      // ------------------------------------------------------------ loads: Q, then K and V
      uint32_t kv = 0, qn = 0;
      uint32_t last_part = 0, parts = 0;  // by stage: whether its last tile went by v_part, and the parity of the next such
      bool ok = true;
      const int per_tile = kRowsT / sh.gs;  // positions of a query tile
      while (ok && run.next(sh, start)) {
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(q_empty, (qn & 1) ^ 1, abort, st, 0xF01)))) break;
        const int g = run.unit / sh.RG, rg = run.unit % sh.RG;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, (uint32_t)((two ? 2 : 1) * L::TILE));
          for (int q = 0; q < (two ? 2 : 1); ++q)
#pragma unroll
            for (int c = 0; c < L::NC; ++c)
              tma_load_3d(sb + q * L::TILE + c * L::CHUNK, &tm_q, c * 64, g * sh.gs, run.seq * sh.T + ((KV4 ? 1 : 2) * rg + q) * per_tile,
                          q_full);
        }
        ++qn;
        __syncwarp();
        if constexpr (KV4) {
          // codes by TMA, a lane a box of the tile; scales, 4 bytes a token, by cp.async, 4 tokens a lane
          const int64_t row0 = (int64_t)run.seq * map.max_pages;
          for (int j = run.t0; ok && j < run.t1; ++j, ++kv) {
            const int rows = min(kKeysT, run.len - j * kKeysT), boxes = (rows + box_rows - 1) / box_rows;
            int32_t row = 0;
            if (lane < boxes) {
              const int t = j * kKeysT + lane * box_rows, lp = t / map.page;
              int32_t pp = __ldg(map.table + row0 + lp);
              if (pp < 0 || (int64_t)pp >= map.n_pages) {
                raise_error(st, kErrBadIndex, 3u);
                pp = 0;
              }
              row = pp * (map.page / box_rows) + (t - lp * map.page) / box_rows;  // in boxes
            }
            const int s = (int)(kv % L::DEPTH);
            const uint32_t to = sb + L::raw_at(two) + s * L::RAW, at = raw_full(s);
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(raw_empty(s), ((kv / L::DEPTH) & 1) ^ 1, abort, st, 0xF02)))) break;
            if (lane == 0) mbar_arrive_expect_tx(at, (uint32_t)(2 * boxes * box_rows * (D / 2)));
            __syncwarp();
            if (lane < boxes) {
              tma_load_4d(to + lane * box_rows * (D / 2), &tm_k, 0, 0, g, row, at);
              tma_load_4d(to + L::CODES + lane * box_rows * (D / 2), &tm_v, 0, 0, g, row, at);
            }
#pragma unroll
            for (int i = 0; i < kKeysT / 32; ++i) {
              const int tt = 32 * i + lane;
              const int64_t token = (int64_t)__shfl_sync(0xffffffffu, row, tt / box_rows) * box_rows + (tt & (box_rows - 1));
              if (tt < rows) {
                cp_async4(to + 2 * L::CODES + tt * kGroups, pool.k_scales + (token * pool.H_kv + g) * kGroups);
                cp_async4(to + 2 * L::CODES + L::SCALES + tt * kGroups, pool.v_scales + (token * pool.H_kv + g) * kGroups);
              }
            }
            cp_async_arrive(at);
          }
          continue;
        }
        const int piece = lane / L::NC, chunk = lane % L::NC;  // a lane's box of a tile
        for (int j = run.t0; ok && j < run.t1; ++j) {
          const int rows = min(kKeysT, run.len - j * kKeysT), boxes = (rows + box_rows - 1) / box_rows;
          const bool mine = piece < boxes;
          int32_t row = 0;
          if (mine) {
            const int64_t t = (int64_t)j * kKeysT + piece * box_rows, lp = t / map.page;
            int32_t pp = __ldg(map.table + (int64_t)run.seq * map.max_pages + lp);
            if (pp < 0 || (int64_t)pp >= map.n_pages) {
              raise_error(st, kErrBadIndex, 3u);
              pp = 0;
            }
            row = (int32_t)((int64_t)pp * map.page + (t - lp * map.page));
          }
#pragma unroll 1
          for (int i = 0; i < 2; ++i) {
            const int s = (int)(kv % L::STAGES);
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(kv_empty(s), ((kv / L::STAGES) & 1) ^ 1, abort, st, 0xF02)))) break;
            const bool part = i && rows < kKeysT;
            const uint32_t to = part ? v_part(s) : kv_full(s);
            if (lane == 0) mbar_arrive_expect_tx(to, (uint32_t)(boxes * L::NC * box_rows * 128));
            last_part = part ? last_part | 1u << s : last_part & ~(1u << s);
            parts ^= (uint32_t)part << s;
            __syncwarp();
            if (mine)
              tma_load_3d(sm_kv + s * L::TILE + chunk * L::CHUNK + piece * box_rows * 128, i ? &tm_v : &tm_k, chunk * 64, g, row, to);
            ++kv;
          }
        }
      }
      if (*abort && lane == 0) {  // let the copies in flight land before the CTA ends
        if (KV4)
          for (uint32_t x = kv > (uint32_t)L::DEPTH ? kv - L::DEPTH : 0; x < kv; ++x)
            mbar_wait(raw_full((int)(x % L::DEPTH)), (x / L::DEPTH) & 1, nullptr, st, 0xFF1);
        else
          for (uint32_t x = kv > (uint32_t)L::STAGES ? kv - L::STAGES : 0; x < kv; ++x) {
            const int s = (int)(x % L::STAGES);
            const bool part = last_part >> s & 1u;
            mbar_wait(part ? v_part(s) : kv_full(s), part ? (parts >> s & 1u) ^ 1u : (x / L::STAGES) & 1, nullptr, st, 0xFF1);
          }
        if (qn) mbar_wait(q_full, (qn - 1) & 1, nullptr, st, 0xFF2);
      }
    } else if (KV4 && warp >= kWarpExpand) {
      // ------------------------------------------------------------ 4-bit codes into bf16 tiles
      // A warp has the same 16 tokens of every tile, a lane half a row of K and of V: codes leave as 16-byte pieces of
      // the swizzled tiles (times 2^-18, see expand8_sub); tokens past the context as zeros.
      constexpr int CB = D / 2, HW = D / 64;  // bytes of a row's codes, 16-byte pieces of half of them
      const int r = (warp - kWarpExpand) * kUnitRows + (lane & 15), half = lane >> 4;
      // piece p of a row is at p ^ (row / 2 % 4) of it (32-byte rows: p ^ (row / 4 % 2)), by TMA's swizzle
      const uint32_t codes_at = sb + L::raw_at(two) + r * CB + (((half * HW) ^ (CB == 64 ? (r >> 1) & 2 : (r >> 2) & 1)) << 4);
      const uint32_t odd = CB == 64 ? (r >> 1) & 1 : 0;  // which of the half row's two pieces comes first
      const uint32_t scales_at = sb + L::raw_at(two) + 2 * L::CODES + r * kGroups + 2 * half;
      // word w of the half row goes to piece w of its 64-channel chunk (d = 128), or 4 half + w (d = 64)
      const uint32_t lane_to = sm_kv + (D == 128 ? half * L::CHUNK : 0) + r * 128 + (((D == 128 ? 0 : 4 * half) ^ (r & 7)) << 4);
      int slot = 0;
      uint32_t raw_ph = 0, ks = 0, kph = 1;  // parities of the ring's next use, of the last use of the next K tile's stage
      bool ok = true;
      while (ok && run.next(sh, start)) {
#pragma unroll 1
        for (int j = run.t0; j < run.t1; ++j) {
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(raw_full(slot), raw_ph, abort, st, 0xF05)))) break;
          uint4 kc[HW], vc[HW];
          const uint32_t at = codes_at + slot * L::RAW;
#pragma unroll
          for (int y = 0; y < HW; ++y) {
            kc[y] = lds_16(at + ((y ^ odd) << 4) * (HW - 1));
            vc[y] = lds_16(at + L::CODES + ((y ^ odd) << 4) * (HW - 1));
          }
          const uint32_t k_sc = lds_2(scales_at + slot * L::RAW), v_sc = lds_2(scales_at + slot * L::RAW + L::SCALES);
          const bool on = r < run.len - j * kKeysT;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(kv_empty(ks), kph, abort, st, 0xF03)))) break;
          expand_half<HW>(kc, k_sc, on, lane_to + ks * L::TILE);
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(kv_empty(ks + 1), kph, abort, st, 0xF04)))) break;
          expand_half<HW>(vc, v_sc, on, lane_to + (ks + 1) * L::TILE);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(raw_empty(slot));
            mbar_arrive(kv_full(ks));
            mbar_arrive(kv_full(ks + 1));
          }
          ks += 2;
          if (ks == (uint32_t)L::STAGES) ks = 0, kph ^= 1u;
          if (++slot == L::DEPTH) slot = 0, raw_ph ^= 1u;
        }
      }
    } else if (!KV4 && warp == kWarpGuard) {
      // ------------------------------------------------------------ guard: rows of V past the context become zeros
      uint32_t kv = 0, parts = 0;
      bool ok = true;
      while (ok && run.next(sh, start)) {
        const int n = run.t1 - run.t0, rows = run.len - (run.t1 - 1) * kKeysT;  // of the last tile
        kv += 2 * n;
        if (rows >= kKeysT) continue;
        const int s = (int)((kv - 1) % L::STAGES);
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(v_part(s), parts >> s & 1u, abort, st, 0xF20)))) break;
        parts ^= 1u << s;
        const uint32_t va = sm_kv + s * L::TILE + (lane & 7) * 16;
        for (int r = rows + (lane >> 3); r < kKeysT; r += 4)
#pragma unroll
          for (int c = 0; c < L::NC; ++c) sts_16(va + c * L::CHUNK + r * 128, make_uint4(0u, 0u, 0u, 0u));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(kv_full(s));
      }
    }
  } else if (warp >= kWarpMma) {
    // -------------------------------------------------------------- products: warp kWarpMma + q for stream q
    // The whole warp runs the loops on warp-uniform values and one elected lane issues.  A wait that gives up is not
    // looked at: the later ones return at once, and every address stays in bounds.
    const int q = (int)uniform((uint32_t)(warp - kWarpMma));
    const uint32_t ts = uniform(tmem) + q * 128, to = ts + L::TMEM_O, lead = elect_one();
    uint32_t ks = 0, kph = 0;          // stage of the next K tile and the parity of its use
    uint32_t sp = 0, ip = 0, qp = 0;   // parities: softmax results, segments with products, query tiles
    const uint64_t qd = umma_desc_kmajor(sb + (two ? q : 0) * L::TILE, 128);
    while (run.next(sh, start)) {
      const int n = (int)uniform((uint32_t)(run.t1 - run.t0));
      const bool any = uniform((uint32_t)(rows_of(run.unit, q) > 0));
      auto on = [&](int j) { return two ? any : (j & 1) == q; };
      const int last = two ? (any ? n - 1 : -1) : n - 1 - ((n - 1 - q) & 1);  // the stream's last tile (below 0: none)
      mbar_wait(q_full, qp, abort, st, 0xF10);
      qp ^= 1u;
      if (last < 0) commit_if(lead, q_empty);
      auto product_s = [&](int j) {
        mbar_wait(kv_full(ks), kph, abort, st, 0xF11);  // (a tile of the other stream too: the ring is walked in step)
        if (on(j)) {
          tc_fence_after();
          const uint64_t kd = umma_desc_kmajor(sm_kv + ks * L::TILE, 128);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * L::CHUNK + (k & 3) * 32) / 16;
            mma_ss_if(lead, ts, qd + off, kd + off, IDESC_S, k > 0);
          }
          commit_if(lead, s_full(q));
          commit_if(lead & (uint32_t)(j == last), q_empty);
        }
        commit_if(lead, kv_empty(ks));
      };
      product_s(0);
      for (int j = 0; j < n; ++j) {
        const uint32_t vs = ks + 1, vph = kph;
        ks += 2;  // the K tile of j + 1
        if (ks == (uint32_t)L::STAGES) ks = 0, kph ^= 1u;
        mbar_wait(kv_full(vs), vph, abort, st, 0xF13);
        if (on(j)) {
          const uint64_t vd = umma_desc_mnmajor_sw128(sm_kv + vs * L::TILE, L::CHUNK);
          const bool first = two ? j == 0 : j < 2;
          if (first) mbar_wait(o_empty(q), ip ^ 1u, abort, st, 0xF15);
          mbar_wait(p_full(q), sp, abort, st, 0xF16);
          sp ^= 1u;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kKeysT / 16; ++k)
            mma_ts_if(lead, to, ts + 32 * (k >> 1) + 8 * (k & 1), vd + k * (16 * 128 / 16), IDESC_PV, (!first || k > 0) ? 1u : 0u);
          commit_if(lead, pv_done(q));
          commit_if(lead & (uint32_t)(j == last), o_full(q));
        }
        commit_if(lead, kv_empty(vs));
        if (j + 1 < n) product_s(j + 1);
      }
      ip ^= (uint32_t)(last >= 0);
    }
    if (*abort) {  // the products in flight end before TMEM is released
      commit_if(lead, drain(q));
      mbar_wait(drain(q), 0, nullptr, st, 0xFF3);
    }
  } else {
    // -------------------------------------------------------------- softmax: keys 32 part .. + 31 of a tile
    if (KV4) regs_inc<80>();
    constexpr int PK = kKeysT / 4, PD = D / 4;
    const int part = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t scol0 = tmem + ((uint32_t)(quarter * 32) << 16) + part * PK;
    const uint32_t ocol0 = tmem + ((uint32_t)(quarter * 32) << 16) + L::TMEM_O + part * PD;
    const float kInf = __int_as_float(0x7f800000);
    const uint64_t sc2 = f2_pack(scale_log2, scale_log2);
    // What a segment's tiles do not need waits in shared memory (a register spilled here costs a trip to L2 each tile:
    // next to 227 KB of shared memory the L1 keeps nothing).  What is kept for each stream still lies in local memory over a
    // 4-bit cache, 48 bytes a thread: 4 loads and a store a warp and tile by its counters, of some 430 instructions.
    runs_s[warp] = run;
    // bits q: parity of stream q's next S; 2 + q: of its next finished segment; 4: buffer of the next exchange
    uint32_t ph = 0;
    auto mx_at = [&](uint32_t i) { return sm_misc + L::MAXIMA + (i * 128 + row) * 16; };
    auto sum_at = [&](int q) { return sm_misc + L::SUMS + (q * 128 + row) * 16; };
    // (A wait that gave up is not looked at: the later ones return at once, and the warps of a quarter stay in step.)
    for (;;) {
      int n, seen, rows[2];  // tiles of the segment, tokens of it, rows of the streams
      {
        Run r = runs_s[warp];
        if (!r.next(sh, start)) break;
        n = r.t1 - r.t0;
        seen = r.len - r.t0 * kKeysT;
        rows[0] = rows_of(r.unit, 0);
        rows[1] = rows_of(r.unit, 1);
        __syncwarp();
        if (lane == 0) runs_s[warp] = r;
        __syncwarp();
      }
      float m[2] = {-kInf, -kInf};
      uint64_t l2[2] = {0, 0};
      for (int j = 0; j < n; ++j) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (two ? rows[q] == 0 : (j & 1) != q) continue;
          if (quarter >= live_q[q]) continue;
          mbar_wait(s_full(q), ph >> q & 1u, abort, st, 0xF40);
          ph ^= 1u << q;
          __syncwarp();
          if (quarter * 32 >= rows[q]) {  // no rows in this unit
            if (lane == 0) mbar_arrive(p_full(q));
            continue;
          }
          tc_fence_after();
          uint32_t x[32];
          tmem_ld_x32(scol0 + q * 128, x);
          tmem_ld_wait();
          reg_fence32(x);
          const int lim = seen - j * kKeysT - part * PK;  // columns that are context
          if (lim < PK) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= lim) x[e] = 0xff800000u;
          }
          float m4[4] = {-kInf, -kInf, -kInf, -kInf};
#pragma unroll
          for (int e = 0; e < 32; e += 2) m4[(e >> 1) & 3] = max3(m4[(e >> 1) & 3], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          // two buffers: who writes one again has met the other warps since they read it
          const uint32_t mx = mx_at(ph >> 4 & 1u);
          ph ^= 16u;
          asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(mx + 4 * part), "f"(fmaxf(max3(m4[0], m4[1], m4[2]), m4[3])) : "memory");
          quarter_sync(quarter);
          const uint4 mo = lds_16(mx);
          const float mt = fmaxf(max3(__uint_as_float(mo.x), __uint_as_float(mo.y), __uint_as_float(mo.z)), __uint_as_float(mo.w)) * scale_log2;
          const bool grow = mt > m[q] + kLazy;  // the threads of a row decide alike
          if (__any_sync(0xffffffffu, grow)) {
            const float alpha = !grow ? 1.f : ex2_approx(m[q] - mt);  // 2^-inf = 0 at the first tile
            if (grow) m[q] = mt;
            float a, b;
            f2_unpack(l2[q], a, b);
            l2[q] = f2_pack(a * alpha, b * alpha);
            if (two ? j > 0 : j > 1) {  // O holds the stream's products so far; this part's columns of it
              mbar_wait(pv_done(q), ph >> q & 1u, abort, st, 0xF41);  // (ph has this S's parity flipped)
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < PD / 16; ++c) {
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
        }
      }
      // ---- the segment's partial result: with one query tile the two streams' merged
      const int nq[2] = {two ? (rows[0] ? n : 0) : (n + 1) / 2, two ? (rows[1] ? n : 0) : n / 2};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (nq[q] == 0 || quarter >= live_q[q]) continue;
        mbar_wait(o_full(q), ph >> (2 + q) & 1u, abort, st, 0xF50);
        __syncwarp();
        ph ^= 4u << q;
        if (quarter * 32 >= rows[q]) continue;
        float a, b;
        f2_unpack(l2[q], a, b);
        asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(sum_at(q) + 4 * part), "f"(a + b) : "memory");
      }
      tc_fence_after();
      const bool alive = quarter * 32 < rows[0] || (two && quarter * 32 < rows[1]);
      if (alive) quarter_sync(quarter);  // (a row of tile 1 has one of tile 0 beside it)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (!two && q == 1) break;
        if (nq[q] == 0 || quarter * 32 >= rows[q]) continue;
        const bool both = !two && nq[1] > 0;
        const uint4 s0 = lds_16(sum_at(q));
        float M = m[q], sum = (__uint_as_float(s0.x) + __uint_as_float(s0.y)) + (__uint_as_float(s0.z) + __uint_as_float(s0.w));
        float w0 = 1.f, w1 = 0.f;  // (4-bit values came in times 2^-18)
        if (both) {
          const uint4 s1 = lds_16(sum_at(1));
          M = fmaxf(m[0], m[1]);
          w0 = m[0] == M ? 1.f : ex2_approx(m[0] - M);
          w1 = m[1] == M ? 1.f : ex2_approx(m[1] - M);
          sum = sum * w0 + ((__uint_as_float(s1.x) + __uint_as_float(s1.y)) + (__uint_as_float(s1.z) + __uint_as_float(s1.w))) * w1;
        }
        if (KV4) w0 *= kSubUnscale, w1 *= kSubUnscale;
        const bool live = row < rows[q];
        const Run& r = runs_s[warp];
        const int64_t slot = (((int64_t)r.seq + r.group) * (sh.H_kv * sh.RG) + r.unit) * sh.RU;
        const int lr = (two ? q * kRowsT : 0) + row;
        float* po = w.part_o + slot * D + part_at(sh.RU, lr, part * PD);
#pragma unroll 1
        for (int c = 0; c < PD / 16; ++c) {
          uint32_t o[16], p[16];
          tmem_ld_x16(ocol0 + q * 128 + c * 16, o);
          tmem_ld_x16(ocol0 + (two ? q : 1) * 128 + c * 16, p);
          tmem_ld_wait();
          reg_fence16(o);
          reg_fence16(p);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            o[e] = __float_as_uint(fmaf(__uint_as_float(o[e]), w0, both ? __uint_as_float(p[e]) * w1 : 0.f));
          if (live)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<float4*>(po + part_at(sh.RU, 0, c * 16 + 4 * e)) =
                  make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                              __uint_as_float(o[4 * e + 3]));
        }
        if (live && part == 0) w.part_ml[slot + lr] = make_float2(M, sum);
      }
      tc_fence_before();
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (nq[q] && quarter < live_q[q] && lane == 0) mbar_arrive(o_empty(q));
    }
  }

  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0) w.errors[blockIdx.x] = est[0];
}

// ---------------------------------------------------------------- the drafts' own part, and joining the partials
// A CTA has 16 to 64 rows (node, head) of a (sequence, K/V head).  The drafts' K and V go to shared memory as bf16; a warp
// for each 16 rows works out their softmax over the drafts that they see with mma.sync (m16n8k16; rows of T gs and at most 64
// keys do not fill a tcgen05 tile).  Then, once the context kernel has ended, a warp for two rows joins that with the rows'
// partials, four of each in flight.  Where there are few rows, up to 16 CTAs share those of a tile, and the warps of a CTA a
// row.  Measured, 16 trees of 64 nodes, 32768 rows, with a cold L2: 31 us, of which the launch's instructions are
// half (46 with one row in hand, one piece of K or V in flight and CTAs of 256 threads; 70 with a warp a row for the drafts
// too, key by key in fp32).
// V's values that are not finite are taken out of shared memory, so that a weight of 0 leaves them out, and added for the rows
// that see them.
template <int D>
struct JoinLayout {
  static constexpr int ROW = D * 2, KV = kMaxT * ROW;  // bytes of a head row, of the drafts' K or V
  // O of the drafts takes the place of K and V once they are done with
  __host__ __device__ static constexpr int ml_at(int tiles) { return 2 * KV > tiles * 16 * D * 4 ? 2 * KV : tiles * 16 * D * 4; }
  __host__ __device__ static constexpr int smem(int tiles) { return ml_at(tiles) + tiles * 16 * 8; }
};

template <int D, bool KV4>
__global__ void __launch_bounds__(kJoinThreads, 4) tree_join_kernel(TreeShape sh, const int32_t* __restrict__ parents,
                                                                    const uint16_t* __restrict__ qp, const uint16_t* __restrict__ k_pool,
                                                                    const uint16_t* __restrict__ v_pool, Kv4Pool pool, CacheMap map,
                                                                    int n_cta, int m_tiles, float scale_log2, TreeScratch w,
                                                                    uint16_t* __restrict__ out, float* __restrict__ lse, DeviceStatus* st) {
  using J = JoinLayout<D>;
  constexpr int V = D / 32, CH = D / 8;  // channels of a lane when a row is joined, 16-byte pieces of a row
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ int64_t at[kMaxT];  // head rows of the drafts
  __shared__ uint64_t sees[kMaxT];
  __shared__ int up[2][kMaxT];
  __shared__ __align__(16) float more_o[kJoinWarps][D];  // of rows that several warps share
  __shared__ float2 more_ml[kJoinWarps];
  __shared__ int bad_s;
  __shared__ unsigned long long wild_s;  // drafts whose V holds values that are not finite
  float* o_s = reinterpret_cast<float*>(sm);                             // [16 m_tiles][D]
  float2* ml_s = reinterpret_cast<float2*>(sm + J::ml_at(m_tiles));  // [16 m_tiles]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / sh.H_kv, g = blockIdx.x % sh.H_kv;
  const int r_cta = blockIdx.y * 16 * m_tiles;  // the CTA's first row
  int n, T;
  bool bad = !sh.lengths(b, n, T);
  if (tid == 0) bad_s = 0, wild_s = 0ull;
  if (tid < kMaxT) {
    sees[tid] = 0;
    up[0][tid] = -1;
    if (tid < T) {
      int p = parents[(int64_t)b * sh.T + tid];
      if (p < -1 || p >= tid) bad = true, p = -1;
      up[0][tid] = p;
      sees[tid] = 1ull << tid;
      const int64_t t = (int64_t)n + tid, lp = t / map.page;
      int32_t pp = __ldg(map.table + (int64_t)b * map.max_pages + lp);
      if (pp < 0 || (int64_t)pp >= map.n_pages) bad = true, pp = 0;
      at[tid] = ((int64_t)pp * map.page + (t - lp * map.page)) * sh.H_kv + g;
    }
  }
  if (__syncthreads_or(bad) && g == 0 && blockIdx.y == 0 && blockIdx.z == 0 && tid == 0) bad_s = 1;
  // ---- K and V of the drafts, 16-byte pieces: K's piece x of row r at x ^ 4 (r & 1), V's at x ^ (r & 7); rows past T are zeros
  const int Tp = (T + 15) & ~15;
  constexpr int FLY = 4;  // pieces of a thread in flight
  for (int x0 = tid; x0 < 2 * Tp * CH; x0 += FLY * kJoinThreads) {
    uint4 raw[FLY];
#pragma unroll
    for (int f = 0; f < FLY; ++f) {
      const int x = x0 + f * kJoinThreads;
      const bool is_v = x >= Tp * CH;
      const int y = is_v ? x - Tp * CH : x, r = y / CH, ch = y % CH;
      raw[f] = make_uint4(0u, 0u, 0u, 0u);
      if (x < 2 * Tp * CH && r < T) {
        const int64_t hr = at[r];
        if constexpr (!KV4) {
          raw[f] = *reinterpret_cast<const uint4*>((is_v ? v_pool : k_pool) + hr * D + ch * 8);
        } else {
          raw[f].x = reinterpret_cast<const uint32_t*>((is_v ? pool.v_codes : pool.k_codes) + hr * (D / 2))[ch];
          raw[f].y = (is_v ? pool.v_scales : pool.k_scales)[hr * kGroups + ch / (CH / kGroups)];
        }
      }
    }
#pragma unroll
    for (int f = 0; f < FLY; ++f) {
      const int x = x0 + f * kJoinThreads;
      if (x >= 2 * Tp * CH) break;
      const bool is_v = x >= Tp * CH;
      const int y = is_v ? x - Tp * CH : x, r = y / CH, ch = y % CH;
      uint4 c = raw[f];
      if (KV4 && r < T) {
        const uint32_t s1 = scale_bf16(c.y), s2 = s1 | (s1 << 16);
        c = expand8(c.x, s2, scale_bias(s2));
      }
      if (is_v) {
        uint32_t v[4] = {c.x, c.y, c.z, c.w};
        const uint32_t top = __vmaxu2(__vmaxu2(v[0] & 0x7FFF7FFFu, v[1] & 0x7FFF7FFFu), __vmaxu2(v[2] & 0x7FFF7FFFu, v[3] & 0x7FFF7FFFu));
        if (top >= 0x7F800000u || (top & 0xFFFFu) >= 0x7F80u) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if ((v[j] & 0x7F80u) == 0x7F80u) v[j] &= 0xFFFF0000u;
            if ((v[j] & 0x7F800000u) == 0x7F800000u) v[j] &= 0x0000FFFFu;
          }
          atomicOr(&wild_s, 1ull << r);
          c = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
      *reinterpret_cast<uint4*>(sm + (is_v ? J::KV : 0) + r * J::ROW + ((ch ^ (is_v ? r & 7 : (r & 1) << 2)) << 4)) = c;
    }
  }
  // who is above whom, in doubling steps
  for (int i = 0, far = 1; far < T; far <<= 1, i ^= 1) {
    uint64_t s = 0;
    int u = -1;
    if (tid < T) {
      u = up[i][tid];
      if (u >= 0) {
        s = sees[u];
        u = up[i][u];
      }
    }
    __syncthreads();
    if (tid < T) {
      sees[tid] |= s;
      up[i ^ 1][tid] = u;
    }
    __syncthreads();
  }
  __syncthreads();
  const float kInf = __int_as_float(0x7f800000);
  const int rows = T * sh.gs;
  const int64_t first_row = (int64_t)b * sh.T * (sh.H_kv * sh.gs) + g * sh.gs;  // row r is first_row + (r / gs) H_q + r % gs
  const int H_q = sh.H_kv * sh.gs, lg = __ffs(sh.gs) - 1;  // (gs is a power of two)
  const bool drafts = warp < m_tiles && r_cta + warp * 16 < rows;  // (the warp's)
  float own_o[D / 8][4], own_m[2], own_l[2];  // O, maxima and sums of a lane's part of its two rows
  if (drafts) {
    // ---- 16 rows over the drafts: a lane has rows lane / 4 and 8 more, channels and keys by lane % 4
    const int r = lane >> 2, c = lane & 3;
    own_m[0] = own_m[1] = -kInf;
    own_l[0] = own_l[1] = 0.f;
    uint32_t qf[2][D / 8];  // channels 8 (4 t + c) .. + 7 of both rows: two steps of 16 each
    uint64_t mask[2], seen[2];  // drafts that a row sees, and from this lane's first key on
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = r_cta + warp * 16 + r + 8 * e;
      mask[e] = rr < rows ? sees[rr >> lg] : 0ull;
      seen[e] = mask[e] >> (2 * c);
      const uint16_t* p = qp + (first_row + (int64_t)(rr >> lg) * H_q + (rr & (sh.gs - 1))) * D;
#pragma unroll
      for (int t = 0; t < D / 32; ++t) {
        const uint4 y = rr < rows ? *reinterpret_cast<const uint4*>(p + (4 * t + c) * 8) : make_uint4(0u, 0u, 0u, 0u);
        qf[e][4 * t] = y.x, qf[e][4 * t + 1] = y.y, qf[e][4 * t + 2] = y.z, qf[e][4 * t + 3] = y.w;
      }
    }
    float s[kMaxT / 8][4];
#pragma unroll
    for (int j = 0; j < kMaxT / 8; ++j) {
      s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
      if (8 * j < Tp) {
        const uint8_t* kr = sm + (8 * j + r) * J::ROW;
#pragma unroll
        for (int t = 0; t < D / 32; ++t) {
          const uint4 y = *reinterpret_cast<const uint4*>(kr + (((4 * t + c) ^ ((r & 1) << 2)) << 4));
          const uint32_t a0[4] = {qf[0][4 * t], qf[1][4 * t], qf[0][4 * t + 1], qf[1][4 * t + 1]}, b0[2] = {y.x, y.y};
          const uint32_t a1[4] = {qf[0][4 * t + 2], qf[1][4 * t + 2], qf[0][4 * t + 3], qf[1][4 * t + 3]}, b1[2] = {y.z, y.w};
          mma_bf16_16816(s[j], a0, b0);
          mma_bf16_16816(s[j], a1, b1);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const bool on = seen[x >> 1] >> (8 * j + (x & 1)) & 1ull;
          s[j][x] = on ? s[j][x] * scale_log2 : -kInf;
          own_m[x >> 1] = fmaxf(own_m[x >> 1], s[j][x]);
        }
      }
    }
    float mz[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      own_m[e] = fmaxf(own_m[e], __shfl_xor_sync(0xffffffffu, own_m[e], 1));
      own_m[e] = fmaxf(own_m[e], __shfl_xor_sync(0xffffffffu, own_m[e], 2));
      mz[e] = own_m[e] == -kInf ? 0.f : own_m[e];  // scores of -inf alone weigh 0
    }
#pragma unroll
    for (int j = 0; j < D / 8; ++j) own_o[j][0] = own_o[j][1] = own_o[j][2] = own_o[j][3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < kMaxT / 16; ++kk) {
      if (16 * kk >= Tp) break;
      uint32_t pa[4];  // weights of 16 keys: row r, row r + 8, each keys 2 c and 8 more
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p0 = ex2_approx(s[2 * kk + y][2 * e] - mz[e]), p1 = ex2_approx(s[2 * kk + y][2 * e + 1] - mz[e]);
          own_l[e] += p0 + p1;
          pa[2 * y + e] = pack_bf16x2(p0, p1);
        }
      const int vr = 16 * kk + (lane & 15);
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t v[4];
        ldmatrix_x4_trans(v[0], v[1], v[2], v[3], sm + J::KV + vr * J::ROW + (((2 * j + (lane >> 4)) ^ (vr & 7)) << 4));
        const uint32_t b0[2] = {v[0], v[1]}, b1[2] = {v[2], v[3]};
        mma_bf16_16816(own_o[2 * j], pa, b0);
        mma_bf16_16816(own_o[2 * j + 1], pa, b1);
      }
    }
    if (wild_s) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        for (uint64_t left = mask[e] & wild_s; left; left &= left - 1) {
          const int64_t hr = at[__ffsll((long long)left) - 1];
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int ch = 8 * j + 2 * c + x;
              float v;
              if constexpr (KV4) v = pool.v_scales[hr * kGroups + ch / (D / kGroups)] == kScaleNaN ? __uint_as_float(0x7FFFFFFFu) : 0.f;
              else v = __uint_as_float((uint32_t)v_pool[hr * D + ch] << 16);
              if ((__float_as_uint(v) & 0x7F800000u) == 0x7F800000u) own_o[j][2 * e + x] += v;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      own_l[e] += __shfl_xor_sync(0xffffffffu, own_l[e], 1);
      own_l[e] += __shfl_xor_sync(0xffffffffu, own_l[e], 2);
    }
  }
  __syncthreads();  // K and V are done with
  if (drafts) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int lr = warp * 16 + r + 8 * e;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) *reinterpret_cast<float2*>(o_s + lr * D + 8 * j + 2 * c) = make_float2(own_o[j][2 * e], own_o[j][2 * e + 1]);
      if (c == 0) ml_s[lr] = make_float2(own_m[e], own_l[e]);
    }
  }
  __syncthreads();
  griddep_wait();  // the partials
  if (tid == 0 && bad_s) raise_error(st, kErrBadIndex, 13u);
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
    for (int c = tid; c < n_cta; c += kJoinThreads)
      if (w.errors[c]) raise_error(st, w.errors[c], 3u);
  const int64_t per = (int64_t)sh.H_kv * sh.RG * sh.RU;  // rows of partials from one to the next of a row
  int c0 = 0, c1 = -1;                                   // the first and the last partial of the sequence
  if (T > 0 && n > 0) {
    const int64_t quota = w.starts[sh.B], f0 = w.starts[b];
    c0 = (int)(f0 / quota) * sh.ways;
    c1 = (int)((f0 + ((n - 1) >> sh.lg)) / quota) * sh.ways + sh.ways - 1;
  }
  // the CTA's rows are of one unit (groups of rows are multiples of 64): its first one there, its partials
  const int rg = r_cta / sh.RU;
  const int64_t s0 = b * sh.ways * per + (int64_t)(g * sh.RG + rg) * sh.RU;
  // this CTA's slice of the rows; with fewer rows than warps, several warps a row, each with every `share`-th four partials
  const int slice = 16 * m_tiles / gridDim.z, share = slice < kJoinWarps ? kJoinWarps / slice : 1, sub = warp % share;
  const int r_u = r_cta - rg * sh.RU + blockIdx.z * slice;
  constexpr int NR = 2;  // rows that a warp has in hand, side by side (their partials are) where every warp has two
  const bool beside = slice >= NR * kJoinWarps;
  const int apart = beside ? 1 : kJoinWarps / share;
  for (int i = beside ? NR * warp : warp / share; i < slice; i += NR * kJoinWarps / share) {  // (once, where a row has several warps)
    float acc[NR][V], M[NR], sum[NR];
    bool live[NR];
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      const int lr = blockIdx.z * slice + i + k * apart, r = r_cta + lr;
      live[k] = i + k * apart < slice && r < rows;
      M[k] = -kInf, sum[k] = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[k][e] = 0.f;
      if (live[k] && sub == 0) {
        const float2 own = ml_s[lr];
        M[k] = own.x, sum[k] = own.y;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[k][e] = o_s[lr * D + lane * V + e];
      }
    }
    if (!live[0] && share == 1) break;
    for (int c = c0 + 4 * sub; c <= c1; c += 4 * share) {  // four partials of each in flight
      float2 ml[NR][4];
      float x[NR][4][V];
      const int left = c1 - c;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (u > left) break;
        const int64_t s = s0 + (c + u) * per;
#pragma unroll
        for (int k = 0; k < NR; ++k) {
          ml[k][u] = make_float2(-kInf, 0.f);
#pragma unroll
          for (int e = 0; e < V; ++e) x[k][u][e] = 0.f;
          if (live[k]) {
            const int r = r_u + i + k * apart;
            ml[k][u] = w.part_ml[s + r];
            const float* p = w.part_o + s * D + part_at(sh.RU, r, lane * V);
            if constexpr (V == 4) {
              const float4 y = *reinterpret_cast<const float4*>(p);
              x[k][u][0] = y.x, x[k][u][1] = y.y, x[k][u][2] = y.z, x[k][u][3] = y.w;
            } else {
              const float2 y = *reinterpret_cast<const float2*>(p);
              x[k][u][0] = y.x, x[k][u][1] = y.y;
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        float m = M[k];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (u <= left) m = fmaxf(m, ml[k][u].x);
        const float old = M[k] == m ? 1.f : ex2_approx(M[k] - m);
        sum[k] *= old;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[k][e] *= old;
        M[k] = m;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (u > left) break;
          const float wt = ml[k][u].x == m ? 1.f : ex2_approx(ml[k][u].x - m);
          sum[k] += ml[k][u].y * wt;
#pragma unroll
          for (int e = 0; e < V; ++e) acc[k][e] += x[k][u][e] * wt;
        }
      }
    }
    if (share > 1) {  // the row's warps
      if (sub) {
#pragma unroll
        for (int e = 0; e < V; ++e) more_o[warp][lane * V + e] = acc[0][e];
        if (lane == 0) more_ml[warp] = make_float2(M[0], sum[0]);
      }
      __syncthreads();
      if (sub) break;
      for (int x = 1; x < share; ++x) {
        const float2 ml = more_ml[warp + x];
        const float m = fmaxf(M[0], ml.x), a = M[0] == m ? 1.f : ex2_approx(M[0] - m), wt = ml.x == m ? 1.f : ex2_approx(ml.x - m);
        M[0] = m;
        sum[0] = sum[0] * a + ml.y * wt;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[0][e] = acc[0][e] * a + more_o[warp + x][lane * V + e] * wt;
      }
    }
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      if (!live[k]) continue;
      const int r = r_cta + blockIdx.z * slice + i + k * apart;
      const bool any = sum[k] > 0.f || sum[k] != sum[k];  // scores of -inf alone weigh nothing: out 0, lse -inf
      const float inv = any ? 1.f / sum[k] : 0.f;
      const int64_t row = first_row + (int64_t)(r >> lg) * H_q + (r & (sh.gs - 1));
      uint32_t y[V / 2];
#pragma unroll
      for (int e = 0; e < V / 2; ++e) y[e] = pack_bf16x2(acc[k][2 * e] * inv, acc[k][2 * e + 1] * inv);
      uint32_t* op = reinterpret_cast<uint32_t*>(out + row * D) + lane * (V / 2);
      if constexpr (V == 4) *reinterpret_cast<uint2*>(op) = make_uint2(y[0], y[1]);
      else *op = y[0];
      if (lane == 0 && lse) lse[row] = any ? (M[k] + log2f(sum[k])) * 0.69314718055994530942f : -kInf;
    }
  }
}

size_t carve(const TreePlan& p, char* base, TreeScratch* out) {
  const size_t slots = ((size_t)p.B + p.groups) * p.ways * p.H_kv * p.RG;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* r = base ? base + off : nullptr;
    off += align_up(bytes, 256);
    return r;
  };
  TreeScratch w;
  w.starts = (int64_t*)take(((size_t)p.B + 1) * 8);
  w.errors = (unsigned int*)take((size_t)p.ctas * 4);
  w.part_o = (float*)take(slots * p.RU * p.d * 4);
  w.part_ml = (float2*)take(slots * p.RU * 8);
  if (out) *out = w;
  return off;
}

template <int D, bool KV4>
cudaError_t launch_t(const void* q, const TreePlan& p, const void* k_pool, const void* v_pool, const Kv4Pool& pool,
                     const CacheMap& map, const int32_t* ctx, const int32_t* tree_len, const int32_t* parents, float scale, void* out,
                     float* lse, const TreeScratch& w, DeviceStatus* st, cudaStream_t s) {
  const int gs = p.H_q / p.H_kv, n_cta = p.ctas;
  const float sl2 = scale * 1.4426950408889634f;
  cudaError_t e = cudaSuccess;
  TreeShape sh;
  sh.ctx = ctx;
  sh.tree_len = tree_len;
  sh.cap = map.max_pages * map.page;
  sh.B = p.B;
  sh.T = p.T;
  sh.gs = gs;
  sh.H_kv = p.H_kv;
  sh.RG = p.RG;
  sh.RU = p.RU;
  sh.groups = p.groups;
  sh.rounds = p.rounds;
  sh.ways = p.ways;
  sh.lg = p.few ? few_lg(p.B, sh.cap) : 7;
  static_assert(kKeysT == 1 << 7, "a tile");
  if (p.few) {
    if ((e = launch_tree_few(q, sh, map, pool, D, sl2, w, st, s)) != cudaSuccess) return e;
  } else {
    using L = Layout<D>;
    const bool two = !KV4 && p.T * gs > kRowsT;
    alignas(64) unsigned char tq[128] = {}, tk[128] = {}, tv[128] = {};
    const uint64_t row = (uint64_t)D * 2;
    // q [B T][H_q][d] as boxes {64 channels, gs heads, 128 / gs positions}; pools [rows][H_kv][d] as {64, 1, box_rows}
    int box_rows = 16;
    while (box_rows < kKeysT && map.page % (2 * box_rows) == 0) box_rows *= 2;
    if (!encode_tmap_3d(tq, q, D, (uint64_t)p.H_q, (uint64_t)p.B * p.T, row, (uint64_t)p.H_q * row, 64, gs, kRowsT / gs, 128))
      return cudaErrorInvalidValue;
    if (KV4) {
      // codes [rows][H_kv][d / 2] bytes (as 16-bit words) in the order {word, row of a box, head, box}
      const uint64_t cb = D / 2, boxes = (uint64_t)map.n_pages * (map.page / box_rows);
      const uint64_t dims[4] = {cb / 2, (uint64_t)box_rows, (uint64_t)p.H_kv, boxes};
      const uint64_t strides[3] = {(uint64_t)p.H_kv * cb, cb, (uint64_t)box_rows * p.H_kv * cb};
      const uint32_t box[4] = {(uint32_t)cb / 2, (uint32_t)box_rows, 1, 1};
      if (!encode_tmap_4d(tk, pool.k_codes, dims, strides, box, D / 2) || !encode_tmap_4d(tv, pool.v_codes, dims, strides, box, D / 2))
        return cudaErrorInvalidValue;
    } else {
      const uint64_t rows = (uint64_t)map.n_pages * map.page;
      if (!encode_tmap_3d(tk, k_pool, D, (uint64_t)p.H_kv, rows, row, (uint64_t)p.H_kv * row, 64, 1, box_rows, 128) ||
          !encode_tmap_3d(tv, v_pool, D, (uint64_t)p.H_kv, rows, row, (uint64_t)p.H_kv * row, 64, 1, box_rows, 128))
        return cudaErrorInvalidValue;
    }
    auto kern = tree_context_kernel<D, KV4>;
    // the most that any call needs: another thread's call must not lower it before this one's launch
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::smem(!KV4, KV4));
    if (e != cudaSuccess) return e;
    kern<<<p.ctas, ctx_threads(KV4), L::smem(two, KV4), s>>>(*reinterpret_cast<const CUtensorMap*>(tq), *reinterpret_cast<const CUtensorMap*>(tk),
                                                       *reinterpret_cast<const CUtensorMap*>(tv), sh, map, pool, box_rows,
                                                       KV4 ? sl2 * kSubUnscale : sl2, w, st);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const int R = p.T * gs;
  // tiles of 16 rows a CTA: more than one where that leaves two CTAs an SM
  const int64_t tiles16 = (int64_t)p.B * p.H_kv * ((R + 15) / 16);
  const int sms = num_sms(), m_tiles = tiles16 >= (int64_t)8 * sms ? 4 : tiles16 >= (int64_t)4 * sms ? 2 : 1;
  int slices = 1;  // CTAs that share the joining of 16 rows, where there are few
  while (m_tiles == 1 && slices < 16 && 2 * slices * tiles16 <= 4 * sms) slices *= 2;
  auto join = tree_join_kernel<D, KV4>;
  e = cudaFuncSetAttribute(join, cudaFuncAttributeMaxDynamicSharedMemorySize, JoinLayout<D>::smem(4));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * p.H_kv), (unsigned)((R + 16 * m_tiles - 1) / (16 * m_tiles)), (unsigned)slices);
  cfg.dynamicSmemBytes = JoinLayout<D>::smem(m_tiles);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join, sh, parents, (const uint16_t*)q, (const uint16_t*)k_pool,
                            (const uint16_t*)v_pool, pool, map, n_cta, m_tiles, sl2, w, (uint16_t*)out, lse, st);
}

}  // namespace

TreePlan tree_plan(int B, int T, int H_q, int H_kv, int d, bool kv4) {
  TreePlan p;
  p.B = B;
  p.T = T;
  p.H_q = H_q;
  p.H_kv = H_kv;
  p.d = d;
  const int R = T * (H_q / H_kv);
  p.few = kv4 && R <= kFewRows && H_kv <= kFewHeads;
  if (p.few) {
    p.RG = p.rounds = 1;
    p.RU = R;
    p.ctas = p.groups = few_ctas(R);
    p.ways = few_ways(H_kv);
    return p;
  }
  p.ctas = num_sms();
  p.ways = 1;
  const int most = kv4 ? kRowsT : 2 * kRowsT;
  p.RG = (R + most - 1) / most;
  p.RU = R < most ? R : most;
  // A CTA has one unit (K/V head and row group) and, with the CTAs of the other units of its group, one run of the list
  // of all sequences' tiles.  As many groups as fill the GPU in `rounds` items a CTA; more than one round where one
  // leaves over 7 % of the CTAs without an item.
  const int units = H_kv * p.RG, n_cta = num_sms();
  p.groups = 0;
  for (int k = 1, best = -1; k <= kMaxRounds && best < 93; ++k) {
    const int m = k * n_cta / units, full = 100 * m * units / (k * n_cta);
    if (m >= 1 && full > best) p.groups = m, p.rounds = k, best = full;
  }
  return p;
}

size_t tree_scratch_bytes(const TreePlan& p) { return carve(p, nullptr, nullptr); }

cudaError_t launch_tree(const void* q, const TreePlan& p, const void* k_pool, const void* v_pool, const Kv4Pool* kv4,
                        const CacheMap& map, const int32_t* ctx, const int32_t* tree_len, const int32_t* parents, float scale, void* out,
                        float* lse, void* scratch, DeviceStatus* st, cudaStream_t s) {
  TreeScratch w;
  carve(p, (char*)scratch, &w);
  const Kv4Pool pool = kv4 ? *kv4 : Kv4Pool{};
#define MSA_TREE(D, K) launch_t<D, K>(q, p, k_pool, v_pool, pool, map, ctx, tree_len, parents, scale, out, lse, w, st, s)
  if (kv4) return p.d == 64 ? MSA_TREE(64, true) : MSA_TREE(128, true);
  return p.d == 64 ? MSA_TREE(64, false) : MSA_TREE(128, false);
#undef MSA_TREE
}

}  // namespace msa
