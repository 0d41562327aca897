// Attention of a tree of drafted tokens over a paged cache (msa_tree_decode_paged, msa_tree_decode_paged_kv4).
//
// Node i of sequence b sees the context, tokens 0 .. ctx - 1 of the cache, and of the drafts, tokens ctx + j, those
// with j = i or above it in the tree:  O[b,i,h] = sum_j softmax_j(scale q[b,i,h].k[j,g]) v[j,g].
//
// The two parts are worked out apart, as partial softmaxes (O, maximum, sum).  The context needs no mask: all rows of a
// (sequence, K/V head) see all of it, T gs rows that share every key, a matrix product.  A node's own branch is a
// handful of keys that differ from row to row; the kernel that joins the partials adds it key by key in fp32, and keys
// that a node does not see are never touched, whatever they hold.
//
// The context: the cache is one flat list of 128-token tiles, ordered by (sequence, K/V head, row group, tile); every CTA
// takes an equal run of it, whatever the lengths are.  tree_context_kernel does a tile by tcgen05, S = Q K^T and O += P V
// with 128 query rows, Q and K, V in shared memory, S / P and O in TMEM.  Two streams of it alternate, so that one's
// softmax runs under the other's products:
//   up to 128 rows: one query tile, whose even and odd key tiles are the streams (their O are merged at the run's end);
//   more: two query tiles over the same keys.
// Rows of a tile past the last one are computed on by the tensor cores alone; warps without a row rest.
#include <math.h>

#include "msa_kv4.cuh"
#include "msa_sm100.cuh"

namespace msa {

namespace {

using namespace sm100;
using namespace kv4;

constexpr int kRowsT = 128, kKeysT = 128;
constexpr int kMaxT = 64;  // nodes of a tree: a 64-bit mask
constexpr int kCtxThreads = 768;
constexpr int kWarpMma = 16, kWarpLoad = 18, kWarpGuard = 19;  // 4-bit pages: warps 19 .. 23 expand codes
constexpr int kExpand = 5;                                     // warps that expand codes
constexpr int kUnitRows = 16;                                  // tokens that one of them takes at a time
constexpr int kUnits = kKeysT / kUnitRows;
constexpr int kJoinThreads = 256;
constexpr float kLazy = 8.0f;  // log2 units a row maximum may grow before O is rescaled

struct TreeShape {
  const int32_t* ctx;       // [B]
  const int32_t* tree_len;  // [B], null: T each
  int64_t cap;
  int B, T, gs, H_kv;
  int RG, RU;  // row groups of a (sequence, K/V head), rows of one
  // Nodes and context of sequence b; bad lengths count as none of either.
  __device__ __forceinline__ bool lengths(int b, int& n, int& t) const {
    n = ctx[b];
    t = tree_len ? tree_len[b] : T;
    if (n < 0 || t < 0 || t > T || (int64_t)n + t > cap) {
      n = t = 0;
      return false;
    }
    return true;
  }
  __device__ __forceinline__ int tiles(int b) const {
    int n, t;
    lengths(b, n, t);
    return t ? (int)(((int64_t)n + kKeysT - 1) / kKeysT) : 0;
  }
};

// A CTA's run [f, f1) of the flat list, segment by segment: tiles [t0, t1) of one unit (sequence, head, row group).
struct Run {
  int64_t f, f1, before;  // `before`: tiles before sequence `seq`
  int seq;
  int len, unit, t0, t1;  // of the segment: context length, unit within the sequence
  __device__ __forceinline__ bool next(const TreeShape& sh) {
    if (f >= f1) return false;
    const int units = sh.H_kv * sh.RG;
    for (;;) {  // (ends: f1 is no more than the sum over all sequences)
      const int n = sh.tiles(seq);
      if (f < before + (int64_t)n * units) {
        unit = (int)((f - before) / n);
        const int64_t r0 = before + (int64_t)unit * n;
        t0 = (int)(f - r0);
        t1 = (int)min(f1 - r0, (int64_t)n);
        int t;
        sh.lengths(seq, len, t);
        f += t1 - t0;
        return true;
      }
      before += (int64_t)n * units;
      ++seq;
    }
  }
};

__device__ __forceinline__ int64_t run_quota(int64_t total, int n_cta) { return total ? (total + n_cta - 1) / n_cta : 1; }

template <int D>
struct Layout {
  static constexpr int NC = D / 64;                // 64-channel chunks
  static constexpr int CHUNK = 128 * 128;          // bytes of a chunk of 128 rows
  static constexpr int TILE = NC * CHUNK;
  static constexpr int STAGES = D == 128 ? 4 : 8;  // K and V tiles in flight
  static constexpr int RAW = kUnitRows * D + 2 * kUnitRows * kGroups;  // a unit's codes and scales of K and V
  static constexpr uint32_t TMEM_O = 256;          // S / P of stream q at 128 q, O of stream q at 256 + 128 q
  // places in shared memory, with one or two query tiles
  __host__ __device__ static constexpr int kv_at(bool two) { return (two ? 2 : 1) * TILE; }
  __host__ __device__ static constexpr int misc_at(bool two) { return kv_at(two) + STAGES * TILE; }
  static constexpr int SUMS = 0, MAXIMA = 2 * 128 * 16, BARS = MAXIMA + 2 * 128 * 16, MISC = BARS + 512;
  // units that an expanding warp has in flight: what fits, 8 at most
  __host__ __device__ static constexpr int depth(bool two) {
    const int n = (227 * 1024 - 1024 - 1024 - misc_at(two) - MISC) / (kExpand * RAW);
    return n > 8 ? 8 : n;
  }
  __host__ __device__ static constexpr int smem(bool two, bool kv4) {
    return 1024 + misc_at(two) + MISC + (kv4 ? kExpand * depth(two) * RAW : 0);
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
__device__ __forceinline__ uint32_t lds_4(uint32_t at) {
  uint32_t y;
  asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(y) : "r"(at));
  return y;
}
__device__ __forceinline__ void sts_16(uint32_t at, uint4 y) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
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
// The value that every lane of the warp has, in a uniform register.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// Scratch of a call: what the context kernel leaves for the joining one.
struct TreeScratch {
  int64_t* starts;      // [B + 1] tiles (times units) before each sequence
  unsigned int* errors; // [CTAs] flags each met
  float* part_o;        // [slots][RU][D]; slot = unit + CTA, which no two segments of the flat list share
  float2* part_ml;      // [slots][RU] maximum (log2 units) and sum
};

// `own`: places in the flat list of the CTA's run.  Every thread takes part.  CTA 0 writes starts.
__device__ __forceinline__ void find_run(const TreeShape& sh, int n_cta, int64_t* starts, int64_t* warp_sums, int64_t* found,
                                         Run& run) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = kCtxThreads / 32;
  const int per = (sh.B + kCtxThreads - 1) / kCtxThreads, b0 = min(tid * per, sh.B), b1 = min(b0 + per, sh.B);
  const int64_t units = (int64_t)sh.H_kv * sh.RG;
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += sh.tiles(b);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_sums[warp] = incl;
  if (tid == 0) found[1] = sh.B;
  __syncthreads();
  int64_t total = 0, off = 0;
  for (int w = 0; w < nw; ++w) {
    const int64_t x = warp_sums[w];
    if (w < warp) off += x;
    total += x;
  }
  total *= units;
  const int64_t quota = run_quota(total, n_cta), at = blockIdx.x * quota;
  int64_t x = (off + incl - mine) * units;
  for (int b = b0; b < b1; ++b) {
    const int64_t n = sh.tiles(b) * units;
    if (x <= at && at < x + n) {
      found[0] = x;
      found[1] = b;
    }
    if (blockIdx.x == 0) starts[b] = x;
    x += n;
  }
  if (blockIdx.x == 0 && tid == 0) starts[sh.B] = total;
  __syncthreads();
  run.before = found[0];
  run.seq = (int)found[1];
  run.f = at;
  run.f1 = min(total, at + quota);
}

template <int D, bool KV4>
__global__ void __launch_bounds__(kCtxThreads, 1) tree_context_kernel(
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
  __shared__ int64_t warp_sums[kCtxThreads / 32], found[2];
  DeviceStatus* st = reinterpret_cast<DeviceStatus*>(est);  // the CTA's own (an error touches its first two words)
  const int R = sh.T * sh.gs;
  const bool two = R > kRowsT;  // two query tiles a unit
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
  static_assert(8 * (B0 + 14 + L::STAGES / 2) <= 512, "barriers fit");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();
  // quarters (32 rows) that some tile of a stream uses
  const int most[2] = {min(two ? kRowsT : R, kRowsT), two ? min(sh.RG > 1 ? kRowsT : R - kRowsT, kRowsT) : R};
  const int live_q[2] = {(most[0] + 31) / 32, (most[1] + 31) / 32};
  if (tid == 0) {
    for (int i = 0; i < L::STAGES; ++i) {
      mbar_init(kv_full(i), KV4 ? kUnits : 1);
      mbar_init(kv_empty(i), 2);
    }
    for (int i = 1; i < L::STAGES; i += 2) mbar_init(v_part(i), 1);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
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
    if (!KV4) {
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
    }
  }
  Run run;
  find_run(sh, gridDim.x, w.starts, warp_sums, found, run);
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  volatile int* abort = &abort_flag;
  // rows of query tile q of a unit, and whether stream q takes tile j of the segment
  auto rows_of = [&](int unit, int q) { return min(kRowsT, max(0, R - (unit % sh.RG) * (2 * kRowsT) - (two ? q * kRowsT : 0))); };

  if (warp >= kWarpLoad) {
    if (warp == kWarpLoad) {
      // ------------------------------------------------------------ loads: Q, and bf16 K and V
      uint32_t kv = 0, qn = 0;
      uint32_t last_part = 0, parts = 0;  // by stage: whether its last tile went by v_part, and the parity of the next such
      bool ok = true;
      const int per_tile = kRowsT / sh.gs;  // positions of a query tile
      while (ok && run.next(sh)) {
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(q_empty, (qn & 1) ^ 1, abort, st, 0xF01)))) break;
        const int g = run.unit / sh.RG, rg = run.unit % sh.RG;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, (uint32_t)((two ? 2 : 1) * L::TILE));
          for (int q = 0; q < (two ? 2 : 1); ++q)
#pragma unroll
            for (int c = 0; c < L::NC; ++c)
              tma_load_3d(sb + q * L::TILE + c * L::CHUNK, &tm_q, c * 64, g * sh.gs, run.seq * sh.T + (2 * rg + q) * per_tile,
                          q_full);
        }
        ++qn;
        __syncwarp();
        if (KV4) continue;
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
        if (!KV4)
          for (uint32_t x = kv > (uint32_t)L::STAGES ? kv - L::STAGES : 0; x < kv; ++x) {
            const int s = (int)(x % L::STAGES);
            const bool part = last_part >> s & 1u;
            mbar_wait(part ? v_part(s) : kv_full(s), part ? (parts >> s & 1u) ^ 1u : (x / L::STAGES) & 1, nullptr, st, 0xFF1);
          }
        if (qn) mbar_wait(q_full, (qn - 1) & 1, nullptr, st, 0xFF2);
      }
    } else if (KV4) {
      // ------------------------------------------------------------ 4-bit codes into bf16 tiles
      // A warp takes every kExpand-th unit of 16 tokens: their codes and scales of K and V come by cp.async into its own
      // ring, `depth` units ahead, and leave as 16-byte pieces of the swizzled tiles; tokens past the context as zeros.
      constexpr int CB = D / 2;  // bytes of a head row's codes
      const int wx = warp - kWarpGuard, depth = L::depth(two);
      const uint32_t ring = sm_misc + L::MISC + wx * depth * L::RAW;
      const int row_bytes = pool.H_kv * CB;
      Run ahead = run;
      bool more = ahead.next(sh), have = run.next(sh);
      int au = wx, cu = wx;  // units into the segments
      // the next unit to fetch: false past the last one
      auto settle = [&](Run& r, int& u, bool& on) {
        while (on && u >= (r.t1 - r.t0) * kUnits) {
          u -= (r.t1 - r.t0) * kUnits;
          on = r.next(sh);
        }
      };
      settle(ahead, au, more);
      settle(run, cu, have);
      auto page_of = [&]() {  // page id of the unit that `ahead` stands at (read a unit before it is used)
        const int t = ahead.t0 * kKeysT + au * kUnitRows;
        return more && t < ahead.len ? __ldg(map.table + (int64_t)ahead.seq * map.max_pages + t / map.page) : 0;
      };
      int32_t pp = page_of();
      auto fetch = [&](uint32_t slot) {
        const int t = ahead.t0 * kKeysT + au * kUnitRows;
        if (more && t < ahead.len) {
          if (pp < 0 || (int64_t)pp >= map.n_pages) {
            raise_error(st, kErrBadIndex, 3u);
            pp = 0;
          }
          const int g = ahead.unit / sh.RG;
          const int64_t row = (int64_t)pp * map.page + t % map.page;
          const uint32_t to = ring + slot * L::RAW;
          constexpr int PR = CB / 16;  // 16-byte pieces of a row's codes
#pragma unroll
          for (int i = lane; i < kUnitRows * PR; i += 32) {
            const int r = i / PR, p = i % PR;
            // piece p of row r at p ^ (r / 2 % 4) (64-byte rows; 32-byte rows: p ^ (r / 4 % 2)): conflict-free reads
            const int at = r * CB + ((p ^ (PR == 4 ? (r >> 1) & 3 : (r >> 2) & 1)) << 4);
            const int64_t src = (row + r) * row_bytes + g * CB + p * 16;
            cp_async16(to + at, pool.k_codes + src);
            cp_async16(to + kUnitRows * CB + at, pool.v_codes + src);
          }
          const int r = lane & 15;
          cp_async4(to + 2 * kUnitRows * CB + lane * 4,
                    (lane < 16 ? pool.k_scales : pool.v_scales) + ((row + r) * pool.H_kv + g) * kGroups);
        }
        cp_async_commit();
        au += kExpand;
        settle(ahead, au, more);
        pp = page_of();
      };
      for (int i = 0; i < depth - 1; ++i) fetch(i);
      uint32_t slot = 0, kv0 = 0;  // ring slot; stage index of the segment's first K tile
      bool ok = true;
      while (ok && have) {
        fetch((slot + depth - 1) % depth);
        switch (depth) {
          case 8: cp_async_wait<7>(); break;
          case 7: cp_async_wait<6>(); break;
          case 6: cp_async_wait<5>(); break;
          case 5: cp_async_wait<4>(); break;
          case 4: cp_async_wait<3>(); break;
          case 3: cp_async_wait<2>(); break;
          default: cp_async_wait<1>(); break;
        }
        __syncwarp();
        const int j = cu / kUnits, r0 = (cu % kUnits) * kUnitRows;
        const int left = run.len - (run.t0 + j) * kKeysT - r0;  // tokens of the unit that are context
        const uint32_t from = ring + slot * L::RAW;
        const int r = lane & 15, half = lane >> 4;  // a lane has half a row of K and of V
        const uint32_t kv = kv0 + 2 * j;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int s = (int)((kv + i) % L::STAGES);
          ok = ok && __all_sync(0xffffffffu, mbar_wait(kv_empty(s), (((kv + i) / L::STAGES) & 1) ^ 1, abort, st, 0xF03));
          if (!ok) break;
          const uint32_t codes = from + i * kUnitRows * CB;
          const uint32_t sc = lds_4(from + 2 * kUnitRows * CB + (i * 16 + r) * 4);
          constexpr int NW = D / 16;  // words of half a row
          const uint32_t row_at = sm_kv + s * L::TILE + (r0 + r) * 128;
#pragma unroll
          for (int y = 0; y < NW / 4; ++y) {
            const int p = half * (NW / 4) + y;  // 16-byte piece of the codes
            const uint4 c = lds_16(codes + r * CB + ((p ^ (CB == 64 ? (r >> 1) & 3 : (r >> 2) & 1)) << 4));
            const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int word = 4 * p + x;  // 8 channels; group word / (D / 32)
              const uint32_t b = sc >> (8 * (word / (D / 32))) & 0xFFu, s1 = scale_bf16(b), s2 = s1 | (s1 << 16);
              uint4 v = expand8(cw[x], s2, scale_bias(s2));
              if (r >= left) v = make_uint4(0u, 0u, 0u, 0u);
              sts_16(row_at + (word >> 3) * L::CHUNK + (((word & 7) ^ (r & 7)) << 4), v);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(kv_full(s));
        }
        slot = slot + 1 == (uint32_t)depth ? 0 : slot + 1;
        cu += kExpand;
        while (have && cu >= (run.t1 - run.t0) * kUnits) {
          cu -= (run.t1 - run.t0) * kUnits;
          kv0 += 2 * (run.t1 - run.t0);
          have = run.next(sh);
        }
      }
      cp_async_wait<0>();
    } else if (warp == kWarpGuard) {
      // ------------------------------------------------------------ guard: rows of V past the context become zeros
      uint32_t kv = 0, parts = 0;
      bool ok = true;
      while (ok && run.next(sh)) {
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
    while (run.next(sh)) {
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
    constexpr int PK = kKeysT / 4, PD = D / 4;
    const int part = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t scol0 = tmem + ((uint32_t)(quarter * 32) << 16) + part * PK;
    const uint32_t ocol0 = tmem + ((uint32_t)(quarter * 32) << 16) + L::TMEM_O + part * PD;
    const float kInf = __int_as_float(0x7f800000);
    const uint64_t sc2 = f2_pack(scale_log2, scale_log2);
    uint32_t sn[2] = {0, 0}, in[2] = {0, 0}, ex = 0;  // S products and segments of each stream so far; exchanges
    auto mx_at = [&](uint32_t i) { return sm_misc + L::MAXIMA + (i * 128 + row) * 16; };
    auto sum_at = [&](int q) { return sm_misc + L::SUMS + (q * 128 + row) * 16; };
    // (A wait that gave up is not looked at: the later ones return at once, and the warps of a quarter stay in step.)
    while (run.next(sh)) {
      const int n = run.t1 - run.t0, seg_seq = run.seq, seg_unit = run.unit;
      float m[2] = {-kInf, -kInf};
      uint64_t l2[2] = {0, 0};
      const int rows[2] = {rows_of(run.unit, 0), rows_of(run.unit, 1)};
      for (int j = 0; j < n; ++j) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (two ? rows[q] == 0 : (j & 1) != q) continue;
          if (quarter >= live_q[q]) continue;
          mbar_wait(s_full(q), sn[q] & 1, abort, st, 0xF40);
          __syncwarp();
          if (quarter * 32 >= rows[q]) {  // no rows in this unit
            if (lane == 0) mbar_arrive(p_full(q));
            ++sn[q];
            continue;
          }
          tc_fence_after();
          uint32_t x[32];
          tmem_ld_x32(scol0 + q * 128, x);
          tmem_ld_wait();
          reg_fence32(x);
          const int lim = run.len - (run.t0 + j) * kKeysT - part * PK;  // columns that are context
          if (lim < PK) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= lim) x[e] = 0xff800000u;
          }
          float m4[4] = {-kInf, -kInf, -kInf, -kInf};
#pragma unroll
          for (int e = 0; e < 32; e += 2) m4[(e >> 1) & 3] = max3(m4[(e >> 1) & 3], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          // two buffers: who writes one again has met the other warps since they read it
          const uint32_t mx = mx_at(ex & 1);
          ++ex;
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
              mbar_wait(pv_done(q), (sn[q] - 1) & 1, abort, st, 0xF41);
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
          ++sn[q];
        }
      }
      // ---- the segment's partial result: with one query tile the two streams' merged
      const int64_t slot = (int64_t)seg_seq * (sh.H_kv * sh.RG) + seg_unit + blockIdx.x;
      const int nq[2] = {two ? (rows[0] ? n : 0) : (n + 1) / 2, two ? (rows[1] ? n : 0) : n / 2};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (nq[q] == 0 || quarter >= live_q[q]) continue;
        mbar_wait(o_full(q), in[q] & 1, abort, st, 0xF50);
        __syncwarp();
        ++in[q];
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
        const int other = two ? q : 1;
        const bool both = !two && nq[1] > 0;
        const uint4 s0 = lds_16(sum_at(q));
        float M = m[q], sum = (__uint_as_float(s0.x) + __uint_as_float(s0.y)) + (__uint_as_float(s0.z) + __uint_as_float(s0.w));
        float w0 = 1.f, w1 = 0.f;
        if (both) {
          const uint4 s1 = lds_16(sum_at(1));
          M = fmaxf(m[0], m[1]);
          w0 = m[0] == M ? 1.f : ex2_approx(m[0] - M);
          w1 = m[1] == M ? 1.f : ex2_approx(m[1] - M);
          sum = sum * w0 + ((__uint_as_float(s1.x) + __uint_as_float(s1.y)) + (__uint_as_float(s1.z) + __uint_as_float(s1.w))) * w1;
        }
        const bool live = row < rows[q];
        const int64_t at = slot * sh.RU + (two ? q * kRowsT : 0) + row;
        float4* po = reinterpret_cast<float4*>(w.part_o + at * D + part * PD);
#pragma unroll 1
        for (int c = 0; c < PD / 16; ++c) {
          uint32_t o[16], p[16];
          tmem_ld_x16(ocol0 + q * 128 + c * 16, o);
          if (both) tmem_ld_x16(ocol0 + other * 128 + c * 16, p);
          tmem_ld_wait();
          reg_fence16(o);
          if (both) {
            reg_fence16(p);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * w0 + __uint_as_float(p[e]) * w1);
          }
          if (live)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              po[c * 4 + e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                                          __uint_as_float(o[4 * e + 3]));
        }
        if (live && part == 0) w.part_ml[at] = make_float2(M, sum);
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
// 4 (d = 128) or 2 channels of a cached head row, as a lane of a warp holds them.
template <int D, bool KV4>
struct Row {
  static constexpr int V = D / 32;
  __device__ static __forceinline__ void load(const uint16_t* bf, const uint8_t* codes, const uint8_t* scales, int64_t row, int H_kv,
                                              int g, float (&x)[V]) {
    const int lane = threadIdx.x & 31;
    const int64_t hr = row * H_kv + g;
    if constexpr (!KV4) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(bf + hr * D) + lane * (V / 2);
      if constexpr (V == 4) {
        const uint2 y = *reinterpret_cast<const uint2*>(p);
        x[0] = bf16_lo(y.x), x[1] = bf16_hi(y.x), x[2] = bf16_lo(y.y), x[3] = bf16_hi(y.y);
      } else {
        const uint32_t y = *p;
        x[0] = bf16_lo(y), x[1] = bf16_hi(y);
      }
    } else {
      // channel c of a word sits in nibble c / 2 + 4 (c % 2)
      const uint32_t y = reinterpret_cast<const uint32_t*>(codes + hr * (D / 2))[lane * V / 8] >> (V == 4 ? 8 * (lane & 1) : 4 * (lane & 3));
      const uint32_t b = scales[hr * kGroups + lane / 8];
      const float s = b == kScaleNaN ? __uint_as_float(0x7FFFFFFFu) : scale_f32(b);
      x[0] = (float)((int)(y & 15u) - 8) * s, x[1] = (float)((int)(y >> 16 & 15u) - 8) * s;
      if constexpr (V == 4) x[2] = (float)((int)(y >> 4 & 15u) - 8) * s, x[3] = (float)((int)(y >> 20 & 15u) - 8) * s;
    }
  }
};

// A warp a row (node, head): its partials of the context merged, then the drafts that it sees one after the other.
template <int D, bool KV4>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(TreeShape sh, const int32_t* __restrict__ parents,
                                                                 const uint16_t* __restrict__ qp, const uint16_t* __restrict__ k_pool,
                                                                 const uint16_t* __restrict__ v_pool, Kv4Pool pool, CacheMap map,
                                                                 int n_cta, int rows_per_warp, float scale_log2, TreeScratch w,
                                                                 uint16_t* __restrict__ out, float* __restrict__ lse, DeviceStatus* st) {
  constexpr int V = D / 32;
  __shared__ int64_t at[kMaxT];  // cache rows of the drafts
  __shared__ uint64_t sees[kMaxT];
  __shared__ int up[2][kMaxT];
  __shared__ int bad_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / sh.H_kv, g = blockIdx.x % sh.H_kv;
  int n, T;
  bool bad = !sh.lengths(b, n, T);
  if (tid == 0) bad_s = 0;
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
      at[tid] = (int64_t)pp * map.page + (t - lp * map.page);
    }
  }
  __syncthreads();
  if (bad) bad_s = 1;
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
  griddep_wait();  // the partials
  __syncthreads();
  if (bad_s && g == 0 && blockIdx.y == 0 && tid == 0) raise_error(st, kErrBadIndex, 13u);
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int c = tid; c < n_cta; c += kJoinThreads)
      if (w.errors[c]) raise_error(st, w.errors[c], 3u);
  const int64_t total = w.starts[sh.B], quota = run_quota(total, n_cta);
  const int tiles = sh.tiles(b);
  const int r0 = (blockIdx.y * (kJoinThreads / 32) + warp) * rows_per_warp;
  for (int r = r0; r < r0 + rows_per_warp; ++r) {
    const int i = r / sh.gs, hh = r % sh.gs;
    if (i >= T) break;
    const int64_t row = ((int64_t)b * sh.T + i) * (sh.H_kv * sh.gs) + g * sh.gs + hh;
    float M = -__int_as_float(0x7f800000), Lsum = 0.f, acc[V], q[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(qp + row * D) + lane * (V / 2);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) q[2 * e] = bf16_lo(p[e]) * scale_log2, q[2 * e + 1] = bf16_hi(p[e]) * scale_log2;
    }
    const float kInf = __int_as_float(0x7f800000);
    if (tiles) {
      const int rg = r / sh.RU, unit = g * sh.RG + rg;
      const int64_t f0 = w.starts[b] + (int64_t)unit * tiles, f1 = f0 + tiles;
      const int c0 = (int)(f0 / quota), c1 = (int)((f1 - 1) / quota);
      const int64_t s0 = ((int64_t)b * (sh.H_kv * sh.RG) + unit) * sh.RU + (r - rg * sh.RU);
      for (int c = c0; c <= c1; c += 4) {  // four partials in flight
        float2 ml[4];
        float x[4][V];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          ml[u] = make_float2(-kInf, 0.f);
#pragma unroll
          for (int e = 0; e < V; ++e) x[u][e] = 0.f;
          if (c + u <= c1) {
            const int64_t s = s0 + (int64_t)(c + u) * sh.RU;
            ml[u] = w.part_ml[s];
            const float* p = w.part_o + s * D + lane * V;
            if constexpr (V == 4) {
              const float4 y = *reinterpret_cast<const float4*>(p);
              x[u][0] = y.x, x[u][1] = y.y, x[u][2] = y.z, x[u][3] = y.w;
            } else {
              const float2 y = *reinterpret_cast<const float2*>(p);
              x[u][0] = y.x, x[u][1] = y.y;
            }
          }
        }
        const float m = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
        const float old = M == m ? 1.f : ex2_approx(M - m);
        Lsum *= old;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] *= old;
        M = m;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float wt = ml[u].x == m ? 1.f : ex2_approx(ml[u].x - m);
          Lsum += ml[u].y * wt;
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] += x[u][e] * wt;
        }
      }
    }
    for (uint64_t left = sees[i]; left; ) {  // two drafts at a time
      const int j0 = __ffsll((long long)left) - 1;
      left &= left - 1;
      const bool pair = left != 0;
      const int j1 = pair ? __ffsll((long long)left) - 1 : j0;
      left &= left - 1;
      float k0[V], k1[V], v0[V], v1[V];
      Row<D, KV4>::load(k_pool, pool.k_codes, pool.k_scales, at[j0], sh.H_kv, g, k0);
      Row<D, KV4>::load(k_pool, pool.k_codes, pool.k_scales, at[j1], sh.H_kv, g, k1);
      Row<D, KV4>::load(v_pool, pool.v_codes, pool.v_scales, at[j0], sh.H_kv, g, v0);
      Row<D, KV4>::load(v_pool, pool.v_codes, pool.v_scales, at[j1], sh.H_kv, g, v1);
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) s0 = fmaf(q[e], k0[e], s0), s1 = fmaf(q[e], k1[e], s1);
#pragma unroll
      for (int o = 16; o; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o), s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      if (!pair) s1 = -kInf;
      const float m = fmaxf(M, fmaxf(s0, s1)), mz = m == -kInf ? 0.f : m;  // scores of -inf alone weigh 0
      const float old = M == m ? 1.f : ex2_approx(M - mz), p0 = ex2_approx(s0 - mz), p1 = ex2_approx(s1 - mz);
      Lsum = Lsum * old + (p0 + p1);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = fmaf(p0, v0[e], acc[e] * old);
      if (pair)
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(p1, v1[e], acc[e]);
      M = m;
    }
    const bool any = Lsum > 0.f || Lsum != Lsum;  // scores of -inf alone weigh nothing: out 0, lse -inf
    const float inv = any ? 1.f / Lsum : 0.f;
    uint32_t* op = reinterpret_cast<uint32_t*>(out + row * D) + lane * (V / 2);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) op[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (lane == 0 && lse) lse[row] = any ? (M + log2f(Lsum)) * 0.69314718055994530942f : -kInf;
  }
}

size_t carve(const TreePlan& p, char* base, TreeScratch* out) {
  const size_t units = (size_t)p.B * p.H_kv * p.RG, slots = units + num_sms();
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* r = base ? base + off : nullptr;
    off += align_up(bytes, 256);
    return r;
  };
  TreeScratch w;
  w.starts = (int64_t*)take(((size_t)p.B + 1) * 8);
  w.errors = (unsigned int*)take((size_t)num_sms() * 4);
  w.part_o = (float*)take(slots * p.RU * p.d * 4);
  w.part_ml = (float2*)take(slots * p.RU * 8);
  if (out) *out = w;
  return off;
}

template <int D, bool KV4>
cudaError_t launch_t(const void* q, const TreePlan& p, const void* k_pool, const void* v_pool, const Kv4Pool& pool,
                     const CacheMap& map, const int32_t* ctx, const int32_t* tree_len, const int32_t* parents, float scale, void* out,
                     float* lse, const TreeScratch& w, DeviceStatus* st, cudaStream_t s) {
  using L = Layout<D>;
  const int gs = p.H_q / p.H_kv;
  const bool two = p.T * gs > kRowsT;
  alignas(64) unsigned char tq[128] = {}, tk[128] = {}, tv[128] = {};
  const uint64_t row = (uint64_t)D * 2;
  // q [B T][H_q][d] as boxes {64 channels, gs heads, 128 / gs positions}; pools [rows][H_kv][d] as {64, 1, box_rows}
  int box_rows = 16;
  while (box_rows < kKeysT && map.page % (2 * box_rows) == 0) box_rows *= 2;
  if (!encode_tmap_3d(tq, q, D, (uint64_t)p.H_q, (uint64_t)p.B * p.T, row, (uint64_t)p.H_q * row, 64, gs, kRowsT / gs, 128))
    return cudaErrorInvalidValue;
  if (!KV4) {
    const uint64_t rows = (uint64_t)map.n_pages * map.page;
    if (!encode_tmap_3d(tk, k_pool, D, (uint64_t)p.H_kv, rows, row, (uint64_t)p.H_kv * row, 64, 1, box_rows, 128) ||
        !encode_tmap_3d(tv, v_pool, D, (uint64_t)p.H_kv, rows, row, (uint64_t)p.H_kv * row, 64, 1, box_rows, 128))
      return cudaErrorInvalidValue;
  }
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
  auto kern = tree_context_kernel<D, KV4>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::smem(two, KV4));
  if (e != cudaSuccess) return e;
  const float sl2 = scale * 1.4426950408889634f;
  const int n_cta = num_sms();
  kern<<<n_cta, kCtxThreads, L::smem(two, KV4), s>>>(*reinterpret_cast<const CUtensorMap*>(tq), *reinterpret_cast<const CUtensorMap*>(tk),
                                                     *reinterpret_cast<const CUtensorMap*>(tv), sh, map, pool, box_rows, sl2, w, st);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int R = p.T * gs;
  // a row a warp while that leaves the GPU room
  const int64_t rows = (int64_t)p.B * p.H_kv * R;
  const int rows_per_warp = rows >= (int64_t)n_cta * 8 * 32 ? 4 : 1, per_cta = kJoinThreads / 32 * rows_per_warp;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * p.H_kv), (unsigned)((R + per_cta - 1) / per_cta));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_join_kernel<D, KV4>, sh, parents, (const uint16_t*)q, (const uint16_t*)k_pool,
                            (const uint16_t*)v_pool, pool, map, n_cta, rows_per_warp, sl2, w, (uint16_t*)out, lse, st);
}

}  // namespace

TreePlan tree_plan(int B, int T, int H_q, int H_kv, int d) {
  TreePlan p;
  p.B = B;
  p.T = T;
  p.H_q = H_q;
  p.H_kv = H_kv;
  p.d = d;
  const int R = T * (H_q / H_kv);
  p.RG = (R + 2 * kRowsT - 1) / (2 * kRowsT);
  p.RU = R < 2 * kRowsT ? R : 2 * kRowsT;
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
