// The context of drafted trees over a 4-bit cache where a K/V head has few rows (T gs up to 32), as partial softmaxes.
//
// The sequences' 32-token spans are one list, a CTA has an equal run of it.  As in the dense decode over this cache its 8
// warps take H heads x 8 / H pairs of 16-token units at a time (a step, from a ring that TMA fills), and codes become mma.sync
// m16n8k16 operands in registers:
//   S^T [16 tokens x 8 NT rows] = K q^T,  O^T [d x 8 NT rows] += V^T P^T,
// an expanded K or V operand serving the NT groups of 8 rows.  q's operands lie in shared memory where NT > 1 leaves no
// registers for them.  tcgen05's 128-row tile, for which codes have to be expanded into shared memory by warps that wait
// for one another, takes as long for any number of rows up to 32 (2630 cycles a tile of 128 tokens of a head).
// (With 32 rows and d = 128 the 255 registers leave 4 to 12 bytes in local memory: 2 loads and a store a warp by its counters,
// outside the steps.)
//
// Measured with the join, 8 heads, d = 128, tcgen05's form in brackets: 4 sequences of 2^20 tokens, 8 rows a head 817 us
// (2293; 0.84 of HBM's rate, which bounds it), 16 rows 1094 us (2288), 32 rows 1640 us (2297; 0.42 of HBM: 1806 cycles a tile
// and head, of which the products need 1024; with registers for two warps a scheduler, what is left is latency); 16 sequences
// of 15000 to 30000 tokens, 32, 16, 8 rows 169, 116, 93 us (226, 225, 225); 64 of 250 to 500 tokens, 16 and 4 rows 29, 21 us
// (42, 40); one of 1500 tokens, 32, 16, 4 rows 22, 17, 14 us (20, 17, 17).  The choice is by rows and heads alone: lengths are
// on the device, and the table's width says little of them.  So 32 rows over a short context take 2 us more than they might;
// rows beyond 32 have no registers here (a warp holds all of its head's).
#include <math.h>

#include "msa_kv4_units.cuh"
#include "msa_sm100.cuh"
#include "msa_tree.cuh"

namespace msa {

namespace {

using namespace kv4;
using namespace sm100;

constexpr int kWarpUnits = 2;  // units of a warp's step: with one at a time 32 rows take 1870 us instead of 1640, 16 rows 1420 instead of 1094
// CTAs an SM, its shared memory (16 rows in two CTAs of 128 registers and two stages: 1560 us)
template <int NT>
struct Few {
  static constexpr int CTAS = NT == 1 ? 2 : 1;
  static constexpr int SMEM = (CTAS == 2 ? 112 : 224) * 1024;
};
constexpr float kNone = -3e38f;  // a maximum of no score yet: finite, so that scores of -inf alone weigh 0
// Bytes of a stage: K and V codes of a step's units, then their scales of every head.
__host__ __device__ constexpr int stage_of(int d, int units, int heads, int H_kv) {
  return (2 * units * heads * kUnit * (d / 2) + 2 * units * kUnit * H_kv * kGroups + 1023) / 1024 * 1024;
}
// q's operands: 16 bytes a lane for each 32 channels of 8 rows, by warp
__host__ __device__ constexpr int q_bytes(int d, int nt) { return nt == 1 ? 0 : kDecWarps * nt * (d / 32) * 512; }

__device__ __forceinline__ uint4 lds_16(uint32_t at) {
  uint4 y;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w) : "r"(at));
  return y;
}
__device__ __forceinline__ void sts_16(uint32_t at, uint4 y) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w) : "memory");
}

// A CTA's run of the list of spans (32 tokens), and segment by segment units [u0, u1) of one sequence.
constexpr int kLgUnit = 4;
struct Run {
  int f, f1, before;  // next span, end, spans before sequence `seq` (all spans fit an int)
  int seq, len, u0, u1;
  __device__ __forceinline__ bool next(const TreeShape& sh) {
    if (f >= f1) return false;
    int n, t;
    while (f >= before + (n = sh.spans(seq))) before += n, ++seq;  // (ends: the runs add up to all spans)
    sh.lengths(seq, len, t);
    const int t0 = f - before, t1 = min(f1 - before, n);
    u0 = t0 << (sh.lg - kLgUnit);
    u1 = min(t1 << (sh.lg - kLgUnit), (len - 1) / kUnit + 1);  // (a sequence with spans is not empty)
    f += t1 - t0;
    return true;
  }
};

// The run of the CTA, a multiple of a step's spans where it has as many: shorter ones leave warps idle, but spread a small
// list over more CTAs.  Every thread takes part.  CTA 0 writes starts.
__device__ __forceinline__ Run find_run(const TreeShape& sh, int step, int64_t* starts) {
  __shared__ int64_t sums[kDecWarps];
  __shared__ int seq_s, before_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (sh.B + kDecThreads - 1) / kDecThreads, b0 = min(tid * per, sh.B), b1 = min(b0 + per, sh.B);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += sh.spans(b);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int64_t total = 0, off = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    const int64_t x = sums[w];
    if (w < warp) off += x;
    total += x;
  }
  int64_t quota = max((total + gridDim.x - 1) / gridDim.x, (int64_t)1);
  if (quota > step) quota = quota_of(total, gridDim.x, step);
  const int64_t first = off + incl - mine, at = blockIdx.x * quota;
  if (at >= first && at < first + mine) {  // (nobody where the CTA has no spans)
    int64_t x = first;
    int b = b0, n;
    while (at >= x + (n = sh.spans(b))) x += n, ++b;
    seq_s = b;
    before_s = (int)x;
  }
  if (blockIdx.x == 0) {
    int64_t x = first;
    for (int b = b0; b < b1; ++b) {
      starts[b] = x;
      x += sh.spans(b);
    }
    if (tid == 0) starts[sh.B] = quota;
  }
  __syncthreads();
  Run r;
  r.f = (int)min(at, total);
  r.f1 = (int)min(total, at + quota);
  r.seq = at < total ? seq_s : 0;
  r.before = at < total ? before_s : 0;
  return r;
}

template <int D, int HC, int NT>
__global__ void __launch_bounds__(kDecThreads, Few<NT>::CTAS) tree_few_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const uint16_t* __restrict__ q, Kv4Pool pool,
    CacheMap map, TreeShape sh, float sl2, int stages, TreeScratch w, DeviceStatus* status) {
  constexpr int G = kWarpUnits, TW = kDecWarps / HC, SU = G * TW;  // units of a warp's step; warps that share a head, units of a step
  constexpr int CT = D / 8;                        // channels of a lane's V column
  using X = Tile<D>;
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages];
  __shared__ int abort_flag;
  __shared__ unsigned int est[2];
  DeviceStatus* st = reinterpret_cast<DeviceStatus*>(est);  // the CTA's own (an error touches its first two words)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H_kv = sh.H_kv, H_q = H_kv * sh.gs, R = sh.RU;
  const int stage = stage_of(D, SU, HC, H_kv);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int i) { return bar0 + 8u * i; };                  // TMA -> consumers
  auto empty = [&](int i) { return bar0 + 8u * (kMaxStages + i); };  // consumers (8 warps) -> TMA
  griddep_launch_dependents();  // the joining grid waits for this one's end
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), kDecWarps);
    }
    fence_mbar_init();
    abort_flag = 0;
    est[0] = est[1] = 0u;
    if (blockIdx.x == 0) {
      status->flags = 0u;
      status->first_code = 0u;
    }
  }
  volatile int* abort = &abort_flag;
  Run run = find_run(sh, max(SU >> (sh.lg - kLgUnit), 1), w.starts);
  const float kInf = __int_as_float(0x7f800000);
  constexpr int kV = SU * HC * X::BYTES, kScales = 2 * kV;  // offsets of V's codes and of the scales in a stage
  const int sc_unit = kUnit * H_kv * kGroups, sc_half = sc_unit / 2;

  const int r = lane >> 2, c = lane & 3;
  const int head = warp % HC, tl = warp / HC;
  const bool on = head < H_kv;
  // this lane's places in its tile: K rows perm(r) (and 8 more), V tokens perm(2c) and perm(2c + 1) (and 8 more)
  const int tile = (G * tl * HC + head) * X::BYTES;  // of the warp's first unit; the second one's is HC tiles on
  const int k_at = tile + X::at(X::perm(r), (X::CB / 4) * c);
  const int v_at0 = kV + tile + X::at(X::perm(2 * c), (X::CB / 8) * r);
  const int v_at1 = kV + tile + X::at(X::perm(2 * c + 1), (X::CB / 8) * r);
  const int ks_at = kScales + G * tl * sc_unit + (X::perm(r) * H_kv + head) * kGroups + c;
  const int vs_at0 = kScales + (SU + G * tl) * sc_unit + (X::perm(2 * c) * H_kv + head) * kGroups + (r >> 1);
  const int vs_at1 = kScales + (SU + G * tl) * sc_unit + (X::perm(2 * c + 1) * H_kv + head) * kGroups + (r >> 1);
  const uint32_t q_at = smem_u32(sm) + stages * stage + warp * (NT * (D / 32) * 512) + lane * 16;
  // the ring's next stage and the parity of its use
  int slot = 0;
  uint32_t phase = 0, at = smem_u32(sm);
  const int ahead = stages - 1;  // steps fetched ahead
  bool ok = true;
  uint32_t fetched = 0;  // stages that this warp has filled, and from bit 16 on the parity of the last time
  while (run.next(sh)) {
    const int steps = (run.u1 - run.u0 + SU - 1) / SU;
    // step i into the stage `off` past `slot`
    auto fetch = [&](int i, int off) {
      int fs = slot + off;
      uint32_t fp = phase;
      if (fs >= stages) fs -= stages, fp ^= 1u;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(empty(fs), fp ^ 1u, abort, st, 0xE21)))) return;
      const int u = run.u0 + i * SU + lane;  // lanes 0 .. SU - 1: a unit each
      const int n = min(SU, run.u1 - u + lane);
      if (lane == 0) mbar_arrive_expect_tx(full(fs), (uint32_t)(n * (2 * HC * X::BYTES + 2 * sc_unit)));
      fetched = (fetched & ~(0x10000u << fs)) | 1u << fs | fp << (16 + fs);
      __syncwarp();
      if (lane < n) {
        const uint32_t upp = (uint32_t)map.page / kUnit, lp = (uint32_t)u / upp;
        const int in_page = ((uint32_t)u - lp * upp) * kUnit;
        int32_t pp = __ldg(map.table + (int64_t)run.seq * map.max_pages + lp);
        if (pp < 0 || (int64_t)pp >= map.n_pages) {
          raise_error(st, kErrBadIndex, 3u);
          pp = 0;
        }
        const uint32_t to = smem_u32(sm) + fs * stage;
        // tiles in (unit, head) order; a page holds whole units
        tma_load_4d(to + lane * HC * X::BYTES, &tm_k, 0, in_page, 0, pp, full(fs));
        tma_load_4d(to + kV + lane * HC * X::BYTES, &tm_v, 0, in_page, 0, pp, full(fs));
        const int64_t row = ((int64_t)pp * map.page + in_page) * (H_kv * kGroups);
        bulk_load(to + kScales + lane * sc_unit, pool.k_scales + row, (uint32_t)sc_unit, full(fs));
        bulk_load(to + kScales + (SU + lane) * sc_unit, pool.v_scales + row, (uint32_t)sc_unit, full(fs));
      }
      __syncwarp();
    };
    if (ok && warp < min(ahead, steps)) fetch(warp, warp);
    // q as B fragments: lane (n = r, c) has channels (D / 4) c .. of row 8 t + r
    uint32_t qf[D / 8];  // (NT = 1)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = 8 * t + r;
      const uint16_t* qp = q + (((int64_t)run.seq * sh.T + row / sh.gs) * H_q + head * sh.gs + row % sh.gs) * D + (D / 4) * c;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 y = on && row < R ? reinterpret_cast<const uint4*>(qp)[i] : make_uint4(0u, 0u, 0u, 0u);
        if (NT == 1) qf[4 * i] = y.x, qf[4 * i + 1] = y.y, qf[4 * i + 2] = y.z, qf[4 * i + 3] = y.w;
        else sts_16(q_at + (t * (D / 32) + i) * 512, y);  // (this lane alone reads it)
      }
    }
    // running maximum in log2 units, and the sum
    float o[D / 16][NT][4], z[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      z[t][0] = z[t][1] = kNone;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i][t][0] = o[i][t][1] = o[i][t][2] = o[i][t][3] = 0.f;
    }
    int units = run.u1 - run.u0 - G * tl;  // left from this warp's place in the step on
    int left = (int)(run.len - (int64_t)(run.u0 + G * tl) * kUnit);  // tokens likewise
    for (int i = 0; i < steps; ++i, units -= SU, left -= SU * kUnit) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(full(slot), phase, abort, st, 0xE20));
      if (ok && on && units > 0) {
        // A second unit past the run's end holds whatever lay in the stage: its tokens count as past the length.
        const int seen = units > 1 ? left : min(left, kUnit);
        uint32_t ks2[G][2], vs2[G][2], top = 0;
#pragma unroll
        for (int h = 0; h < G; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t a = at + h * sc_unit + e * sc_half;
            ks2[h][e] = lds_u8(a + ks_at) * 0x00100010u + kSubScaleBias * 0x00010001u;
            vs2[h][e] = lds_u8(a + vs_at1) * 0x00100000u + (lds_u8(a + vs_at0) * 16u + kSubScaleBias * 0x00010001u);
            top = hmax2_bf16(top, hmax2_bf16(ks2[h][e], vs2[h][e]));
          }
        // a scale of 255 came out as a number, larger than any other: NaN instead
        if (__any_sync(0xffffffffu, (top & 0xFFFFu) == kNaNRaw || (top >> 16) == kNaNRaw)) {
#pragma unroll
          for (int h = 0; h < G; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if ((ks2[h][e] & 0xFFFFu) == kNaNRaw) ks2[h][e] = 0x7FFF7FFFu;
              if ((vs2[h][e] & 0xFFFFu) == kNaNRaw) vs2[h][e] |= 0x7FFFu;
              if ((vs2[h][e] >> 16) == kNaNRaw) vs2[h][e] |= 0x7FFF0000u;
            }
        }
        // S^T = K q^T
        float s[G][NT][4];
        uint32_t kw[G][2][D / 32];
#pragma unroll
        for (int h = 0; h < G; ++h) {
#pragma unroll
          for (int e = 0; e < 2; ++e) lds_words(at + k_at + h * HC * X::BYTES + e * 8 * X::CB, kw[h][e]);
#pragma unroll
          for (int t = 0; t < NT; ++t) s[h][t][0] = s[h][t][1] = s[h][t][2] = s[h][t][3] = 0.f;
        }
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          uint4 y[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t)
            y[t] = NT == 1 ? make_uint4(qf[4 * x], qf[4 * x + 1], qf[4 * x + 2], qf[4 * x + 3]) : lds_16(q_at + (t * (D / 32) + x) * 512);
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const uint4 a = expand8_sub(kw[h][0][x], sub_scale(ks2[h][0])), b = expand8_sub(kw[h][1][x], sub_scale(ks2[h][1]));
            const uint32_t a0[4] = {a.x, b.x, a.y, b.y}, a1[4] = {a.z, b.z, a.w, b.w};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint32_t q0[2] = {y[t].x, y[t].y}, q1[2] = {y[t].z, y[t].w};
              mma_bf16_16816(s[h][t], a0, q0);
              mma_bf16_16816(s[h][t], a1, q1);
            }
          }
        }
        if (seen < G * kUnit) {  // tokens past the length: no score, and whatever lies there stays out of V
#pragma unroll
          for (int h = 0; h < G; ++h) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if (X::perm(r) + 16 * h >= seen) s[h][t][0] = s[h][t][1] = -kInf;
              if (X::perm(r) + 16 * h + 8 >= seen) s[h][t][2] = s[h][t][3] = -kInf;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (X::perm(2 * c) + 16 * h + 8 * e >= seen) vs2[h][e] &= 0xFFFF0000u;
              if (X::perm(2 * c + 1) + 16 * h + 8 * e >= seen) vs2[h][e] &= 0x0000FFFFu;
            }
          }
        }
        bool up = false;
        float n[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            n[t][e] = fmaxf(fmaxf(s[0][t][e], s[0][t][2 + e]), fmaxf(s[1][t][e], s[1][t][2 + e]));
            up |= fmaf(n[t][e], sl2, -kLazy) > z[t][e];
          }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int y = 4; y < 32; y <<= 1) n[t][e] = fmaxf(n[t][e], __shfl_xor_sync(0xffffffffu, n[t][e], y));
              const float zn = fmaxf(n[t][e] * sl2, z[t][e]);
              a[e] = ex2_approx(z[t][e] - zn);
              z[t][e] = zn;
              l[t][e] *= a[e];
            }
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              o[x][t][0] *= a[0], o[x][t][2] *= a[0];
              o[x][t][1] *= a[1], o[x][t][3] *= a[1];
            }
          }
        }
        uint32_t pb[G][NT][2];
#pragma unroll
        for (int h = 0; h < G; ++h)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float p0 = ex2_approx(fmaf(s[h][t][0], sl2, -z[t][0])), p1 = ex2_approx(fmaf(s[h][t][1], sl2, -z[t][1]));
            const float p2 = ex2_approx(fmaf(s[h][t][2], sl2, -z[t][0])), p3 = ex2_approx(fmaf(s[h][t][3], sl2, -z[t][1]));
            l[t][0] += p0 + p2;
            l[t][1] += p1 + p3;
            // P^T as a B operand (tokens x rows): the 8 x 8 halves transposed across the warp
            pb[h][t][0] = movmatrix_t(pack_bf16x2(p0, p1));
            pb[h][t][1] = movmatrix_t(pack_bf16x2(p2, p3));
          }
        // O^T += V^T P^T
#pragma unroll
        for (int h = 0; h < G; ++h) {
          uint32_t vw[4][D / 64];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            lds_words(at + h * HC * X::BYTES + ((e & 1) ? v_at1 : v_at0) + (e >> 1) * 8 * X::CB, vw[e]);
          const SubScale sc[2] = {sub_scale(vs2[h][0]), sub_scale(vs2[h][1])};
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            // halves of the same nibbles of two tokens side by side: even channels from the low halves, odd from the high
            uint32_t ev[2], od[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              ev[e] = __byte_perm(vw[2 * e][x], vw[2 * e + 1][x], 0x5410);
              od[e] = __byte_perm(vw[2 * e][x], vw[2 * e + 1][x], 0x7632);
            }
            const uint4 e0 = expand8_sub(ev[0], sc[0]), e1 = expand8_sub(ev[1], sc[1]);
            const uint4 d0 = expand8_sub(od[0], sc[0]), d1 = expand8_sub(od[1], sc[1]);
            const uint32_t a0[4] = {e0.x, d0.x, e1.x, d1.x}, a1[4] = {e0.y, d0.y, e1.y, d1.y};
            const uint32_t a2[4] = {e0.z, d0.z, e1.z, d1.z}, a3[4] = {e0.w, d0.w, e1.w, d1.w};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              mma_bf16_16816(o[4 * x][t], a0, pb[h][t]);
              mma_bf16_16816(o[4 * x + 1][t], a1, pb[h][t]);
              mma_bf16_16816(o[4 * x + 2][t], a2, pb[h][t]);
              mma_bf16_16816(o[4 * x + 3][t], a3, pb[h][t]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(slot));
      // the warps' turns: the stage before this one, once every warp is done with it, takes the step `ahead` on
      if (ok && ((i + ahead) & (kDecWarps - 1)) == warp && i + ahead < steps) fetch(i + ahead, ahead);
      at += stage;
      if (++slot == stages) slot = 0, phase ^= 1u, at = smem_u32(sm);
    }
    // ---- the segment's partial results, a warp's by themselves
    if (on) {
      const int64_t part = ((((int64_t)run.seq + blockIdx.x) * TW + tl) * H_kv + head) * R;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int y = 4; y < 32; y <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], y);
          const int row = 8 * t + 2 * c + e;
          if (row >= R) continue;
          float* po = w.part_o + part * D + part_at(R, row, CT * r);
#pragma unroll
          for (int i = 0; i < D / 16; i += 2)
            *reinterpret_cast<float4*>(po + part_at(R, 0, 2 * i)) =
                make_float4(o[i][t][e] * kSubUnscale, o[i][t][2 + e] * kSubUnscale, o[i + 1][t][e] * kSubUnscale,
                                    o[i + 1][t][2 + e] * kSubUnscale);
          if (r == 0) w.part_ml[part + row] = make_float2(z[t][e] == kNone ? -kInf : z[t][e], l[t][e]);
        }
    }
  }
  if (*abort && lane == 0)  // a wait gave up: let this warp's copies land before the CTA ends
    for (int i = 0; i < stages; ++i)
      if (fetched >> i & 1u) mbar_wait(full(i), fetched >> (16 + i) & 1u, nullptr, st, 0xEF2);
  __syncthreads();
  if (threadIdx.x == 0) w.errors[blockIdx.x] = est[0];
}

int heads_of(int H_kv) { return H_kv > 4 ? 8 : H_kv > 2 ? 4 : H_kv; }  // the power of two that holds them

template <int D, int HC, int NT>
cudaError_t launch_t(const void* q, const TreeShape& sh, const CacheMap& map, const Kv4Pool& pool, float sl2, const TreeScratch& w,
                     DeviceStatus* st, cudaStream_t s) {
  constexpr int CB = D / 2;
  alignas(64) unsigned char tk[128], tv[128];
  // codes [n_pages][page][H_kv][CB] bytes (as 16-bit words) in the order {row, token, head, page}
  const uint64_t dims[4] = {CB / 2, (uint64_t)pool.page, (uint64_t)pool.H_kv, (uint64_t)pool.n_pages};
  const uint64_t strides[3] = {(uint64_t)pool.H_kv * CB, CB, (uint64_t)pool.page * pool.H_kv * CB};
  const uint32_t box[4] = {CB / 2, kUnit, HC, 1};
  if (!encode_tmap_4d(tk, pool.k_codes, dims, strides, box, CB) || !encode_tmap_4d(tv, pool.v_codes, dims, strides, box, CB))
    return cudaErrorInvalidValue;
  const int stage = stage_of(D, kWarpUnits * kDecWarps / HC, HC, pool.H_kv), qb = q_bytes(D, NT);
  const int fit = (Few<NT>::SMEM - 1024 - qb) / stage, stages = fit > kMaxStages ? kMaxStages : fit;
  auto kern = tree_few_kernel<D, HC, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<NT>::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<sh.groups, kDecThreads, 1024 + stages * stage + qb, s>>>(*reinterpret_cast<const CUtensorMap*>(tk),
                                                                  *reinterpret_cast<const CUtensorMap*>(tv), (const uint16_t*)q, pool,
                                                                  map, sh, sl2, stages, w, st);
  return cudaGetLastError();
}

template <int D, int HC>
cudaError_t launch_h(const void* q, const TreeShape& sh, const CacheMap& map, const Kv4Pool& pool, float sl2, const TreeScratch& w,
                     DeviceStatus* st, cudaStream_t s) {
  return sh.RU <= 8 ? launch_t<D, HC, 1>(q, sh, map, pool, sl2, w, st, s)
         : sh.RU <= 16 ? launch_t<D, HC, 2>(q, sh, map, pool, sl2, w, st, s) : launch_t<D, HC, 4>(q, sh, map, pool, sl2, w, st, s);
}

}  // namespace

int few_ctas(int rows) { return num_sms() * (rows <= 8 ? Few<1>::CTAS : rows <= 16 ? Few<2>::CTAS : Few<4>::CTAS); }
int few_ways(int H_kv) { return kDecWarps / heads_of(H_kv); }
// Spans of 32 tokens where a batch's fit an int, else of 128 (whose number the caller has checked).
int few_lg(int B, int64_t cap) { return (cap + 31) / 32 < ((int64_t)1 << 31) / B ? 5 : 7; }

cudaError_t launch_tree_few(const void* q, const TreeShape& sh, const CacheMap& map, const Kv4Pool& pool, int d, float scale_log2,
                            const TreeScratch& w, DeviceStatus* st, cudaStream_t s) {
  const int HC = heads_of(sh.H_kv);
  const float sl2 = scale_log2 * kSubUnscale;
#define MSA_FEW(D, H) launch_h<D, H>(q, sh, map, pool, sl2, w, st, s)
  if (d == 64) return HC == 8 ? MSA_FEW(64, 8) : HC == 4 ? MSA_FEW(64, 4) : HC == 2 ? MSA_FEW(64, 2) : MSA_FEW(64, 1);
  return HC == 8 ? MSA_FEW(128, 8) : HC == 4 ? MSA_FEW(128, 4) : HC == 2 ? MSA_FEW(128, 2) : MSA_FEW(128, 1);
#undef MSA_FEW
}

}  // namespace msa
