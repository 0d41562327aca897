// Rows of K and V into and out of a 4-bit paged cache, and dense decode over it.
#include <math.h>

#include "msa_kv4_units.cuh"
#include "msa_rows.cuh"
#include "msa_sm100.cuh"

namespace msa {

namespace {

using namespace kv4;
using namespace sm100;

// Rows in (store) and out (load): bound by HBM, 2 d bytes of bf16 and d / 2 + 4 of codes and scales a head row, each
// touched once; the store comes near its instructions too (74 % of issue slots: maxima, scale, 8 roundings a thread).
// A CTA takes R x U x tpp packed rows (tokens), tpp = the tokens that 256 threads cover at 8 channels a thread (K's
// head rows, then V's): it looks all of them up first, then has the reads of U x tpp of them in flight at a time.
// R grows up to kRounds where the CTAs still fill the GPU.
// 131072 tokens of 8 heads, d = 128, in and out: 260 us, 5.23 TB/s (0.77 of the measured copy rate); the store alone 144
// us, 4.72 TB/s (0.70), the load 115 us, 5.89 TB/s (0.87); at d = 64 87 us (0.58) and 66 us (0.77).  604 us in and out
// with U = 1, which is no faster for few rows either (48 tokens: 10.3 and 10.2 us, two launches' latency).
constexpr int kUnroll = 4, kRounds = 8;
struct RowTile {
  int per_tok, tpp;
  __host__ __device__ RowTile(int H_kv, int lanes_per_row) {
    per_tok = 2 * H_kv * lanes_per_row;
    tpp = per_tok < kRowThreads ? kRowThreads / per_tok : 1;
  }
};

template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_store_kernel(const uint16_t* __restrict__ k,
                                                                const uint16_t* __restrict__ v, int64_t N, int R, RowMap map,
                                                                Kv4Pool pool, DeviceStatus* st) {
  constexpr int U = kUnroll, LPR = D / 8, LPG = LPR / kGroups;  // threads of a head row, of a group
  __shared__ int64_t rows[U * kRounds * 16];
  const RowTile rt(pool.H_kv, LPR);
  const int half = rt.per_tok / 2;
  const int64_t i0 = (int64_t)blockIdx.x * R * U * rt.tpp;
  look_up(map, N, i0, R * U * rt.tpp, -1, rows, st);
  const int sub = threadIdx.x / rt.per_tok;  // 0 where a token takes the whole CTA
  for (int c = threadIdx.x - sub * rt.per_tok; c < rt.per_tok; c += kRowThreads) {
    const bool on = sub < rt.tpp, is_v = c >= half;
    const int e = is_v ? c - half : c;  // 8-channel piece of the token's K or V
    const uint16_t* src = (is_v ? v : k) + e * 8;
    uint8_t* codes = is_v ? pool.v_codes : pool.k_codes;
    uint8_t* scales = is_v ? pool.v_scales : pool.k_scales;
    const unsigned lanes = ((1u << LPG) - 1u) << (threadIdx.x & 31u & ~(LPG - 1u));  // the group (per_tok holds whole ones)
#pragma unroll 1
    for (int r = 0; r < R; ++r) {
      int64_t row[U];
      uint4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = (r * U + u) * rt.tpp + sub;
        row[u] = on ? rows[t] : -1;
        x[u] = row[u] >= 0 ? ldg_stream_16(src + (i0 + t) * half * 8) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t sb, code;
        encode8<LPG>(x[u], lanes, code, sb);
        if (row[u] >= 0) {
          reinterpret_cast<uint32_t*>(codes)[row[u] * half + e] = code;
          if (e % LPG == 0) scales[row[u] * (pool.H_kv * kGroups) + e / LPG] = (uint8_t)sb;
        }
      }
    }
  }
}

// The same rows back as exact bf16 values; zeros where the row map has no place.
template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_load_kernel(Kv4Pool pool, int64_t N, int R, RowMap map,
                                                               uint16_t* __restrict__ k, uint16_t* __restrict__ v,
                                                               DeviceStatus* st) {
  constexpr int U = kUnroll, LPR = D / 8, LPG = LPR / kGroups;
  __shared__ int64_t rows[U * kRounds * 16];  // pool row, -1: zeros, -2: a row of no sequence
  const RowTile rt(pool.H_kv, LPR);
  const int half = rt.per_tok / 2;
  const int64_t i0 = (int64_t)blockIdx.x * R * U * rt.tpp;
  look_up(map, N, i0, R * U * rt.tpp, -2, rows, st);
  const int sub = threadIdx.x / rt.per_tok;
  if (sub >= rt.tpp) return;
  for (int c = threadIdx.x - sub * rt.per_tok; c < rt.per_tok; c += kRowThreads) {
    const bool is_v = c >= half;
    const int e = is_v ? c - half : c;
    const uint8_t* codes = is_v ? pool.v_codes : pool.k_codes;
    const uint8_t* scales = is_v ? pool.v_scales : pool.k_scales;
    uint16_t* dst = (is_v ? v : k) + e * 8;
#pragma unroll 1
    for (int r = 0; r < R; ++r) {
      uint32_t w[U], sb[U];
      int64_t row[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        row[u] = rows[(r * U + u) * rt.tpp + sub];
        const int64_t at = row[u] < 0 ? 0 : row[u];
        w[u] = __ldg(reinterpret_cast<const uint32_t*>(codes) + at * half + e);
        sb[u] = __ldg(scales + at * (pool.H_kv * kGroups) + e / LPG);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (row[u] == -2) continue;
        const uint32_t s = scale_bf16(sb[u]), s2 = s | (s << 16);
        const uint4 x = expand8(w[u], s2, scale_bias(s2));
        *reinterpret_cast<uint4*>(dst + (i0 + (r * U + u) * rt.tpp + sub) * half * 8) = row[u] < 0 ? make_uint4(0u, 0u, 0u, 0u) : x;
      }
    }
  }
}

// ---------------------------------------------------------------- dense decode
// One query token per sequence against its whole cache.  The caches are read
// as one flat list of 16-token units, ordered by (sequence, head block, unit),
// a head block being HC heads (8, or the power of two that holds H_kv; heads
// past H_kv leave their warps idle); every CTA takes an equal run of it,
// whatever the lengths are.  Its 8 warps work on HC heads x TW = 8 / HC pairs of
// units at a time: a step.  Steps come by TMA
// through a ring (K and V codes of HC heads x 16 tokens in one box each, the
// tokens' scales as one bulk copy each); the warps take turns in looking up a
// step's pages and issuing its copies, which leaves nearly all issue slots to
// expanding codes and needs no registers for a warp of its own.
// A run that covers a (sequence, head block) row whole writes its output; the
// others leave (O, max, sum) partials, at most two a CTA, for the combine.
//
// Per unit and head, with mma.sync m16n8k16 (bf16, fp32 accumulation):
//   S^T [16 tokens x 8 heads of the group] = K q^T: a lane holds one group (a
//     quarter) of the channels of 2 tokens, so one scale each, and the query's
//     fragments take the same channel order;
//   O^T [d x 8 heads] += V^T P^T: a lane holds d / 8 channels of 4 tokens; the
//     16-bit halves of two tokens' words are paired before their nibbles are
//     expanded, which transposes V on the way; P^T comes from S^T by movmatrix.
// S^T's row i is token perm(i) of the unit, chosen so that both the K and the V
// reads of the swizzled tiles fall in distinct banks.
//
// Bound: HBM, (d / 2 + 4) 2 H_kv bytes a token, and close to it the integer
// instructions that expand the codes (ALU 53 %, issue 61 % of the slots).
// mma.sync, not tcgen05: a group's 8 query heads fill an n = 8 tile, where
// tcgen05's 128-row tiles would be 15/16 empty, and codes would have to be
// expanded into shared memory instead of registers.  Measured, 64 heads on 8,
// d = 128: 4 sequences of 2^20 tokens 823 us, 5.5 TB/s (0.82 of the measured
// copy rate); 48 sequences of 1200 to 12000, 32 heads on 8: 84 us, 4.2 TB/s
// (0.62, of which some 10 us are the start and the combine); one of 1500 tokens:
// 10.4 us, a chain of round trips.  More than 8 K/V heads cost more, because each
// head block fetches the scales of all heads and its stages get larger: 4 of
// 65536 tokens with 16, 32, 64 heads 130, 353, 711 us at d = 128 (0.65, 0.48,
// 0.47), 93, 160, 332 us at d = 64 (0.48, 0.56, 0.54); with 8 85 us (0.50).
constexpr int kCombThreads = 256;
constexpr int kDecSmem = 112 * 1024;  // two CTAs an SM

// Units of sequence s (at least one, so that an empty sequence's output is written); a length outside
// [0, cap] counts as 0.
__device__ __forceinline__ int64_t units_of(int32_t len, int64_t cap) {
  return len <= 0 || (int64_t)len > cap ? 1 : ((int64_t)len + kUnit - 1) / kUnit;
}

// The split of the flat unit list, worked out by every CTA from the lengths.
struct FlatSplit {
  int64_t total;   // units over all sequences and head blocks
  int64_t quota;   // units a CTA takes
  int64_t before;  // units (times head blocks) before sequence `seq`
  int seq;         // the sequence that holds this CTA's first unit (B if none)
};

template <int HC>
__device__ __forceinline__ FlatSplit flat_split(const int32_t* ctx_len, int B, int64_t cap, int n_hb) {
  __shared__ int64_t part[kDecWarps], found_before;
  __shared__ int found_seq;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // inclusive sums of n over the CTA, the CTA's sum added to `base`
  auto scan = [&](int64_t n, int64_t& base) {
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int64_t off = base;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const int64_t x = part[w];
      if (w < warp) off += x;
      base += x;
    }
    return off + incl;
  };
  if (tid == 0) found_seq = B;
  FlatSplit f;
  f.total = 0;
  int64_t n = tid < B ? units_of(ctx_len[tid], cap) : 0, incl = scan(n, f.total);
  for (int s = kDecThreads + tid; s - tid < B; s += kDecThreads) {  // more sequences than threads: the sum first
    __syncthreads();  // part is read
    scan(s < B ? units_of(ctx_len[s], cap) : 0, f.total);
  }
  f.total *= n_hb;
  f.quota = quota_of(f.total, gridDim.x, 2 * kDecWarps / HC);
  const int64_t at = blockIdx.x * f.quota;
  int64_t base = 0;
  for (int s = tid;; s += kDecThreads) {
    if (B > kDecThreads) {
      n = s < B ? units_of(ctx_len[s], cap) : 0;
      __syncthreads();  // part is read
      incl = scan(n, base);
    }
    const int64_t lo = (incl - n) * n_hb;
    if (n > 0 && lo <= at && at < incl * n_hb) {
      found_seq = s;
      found_before = lo;
    }
    if (B <= kDecThreads || s - tid + kDecThreads >= B || base * n_hb > at) break;  // uniform
  }
  __syncthreads();
  f.seq = found_seq;
  f.before = found_before;
  return f;
}

// What a CTA leaves beside its partials: the row that it is the second CTA of, if any, and the errors it met.  Every
// CTA writes its own record, so nothing has to be cleared before a call.
struct __align__(16) SplitRow {
  int seq, hb;  // seq -1: no such row
  int c0, c1;   // the CTAs that hold it
  int part0;    // which partial of c0 it is (partial 0 of the others)
  unsigned int flags, first_code;
  int pad;
};

// A CTA's run, segment by segment: units [u0, u1) of the T units of (sequence, head block).
struct Segments {
  const int32_t* ctx_len;
  int64_t cap, f, f1, before;
  int seq, n_hb;
  // the segment
  int64_t len, T, u0, u1;
  int hb;
  bool bad;
  __device__ __forceinline__ bool next() {
    if (f >= f1) return false;
    const int32_t raw = ctx_len[seq];
    bad = raw < 0 || (int64_t)raw > cap;
    len = bad ? 0 : raw;
    T = units_of(raw, cap);
    hb = (int)((f - before) / T);
    const int64_t r0 = before + hb * T;
    u0 = f - r0;
    u1 = min(f1 - r0, T);
    return true;
  }
  __device__ __forceinline__ void done() {
    f += u1 - u0;
    if (f >= before + n_hb * T) {
      before += n_hb * T;
      ++seq;
    }
  }
};

template <int D, int HC>
__global__ void __launch_bounds__(kDecThreads, 2) kv4_dense_decode_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const uint16_t* __restrict__ q,
    Kv4Pool pool, CacheMap map, const int32_t* __restrict__ ctx_len, int B, int64_t cap, int gs, float scale, int stages,
    uint16_t* __restrict__ out, float* __restrict__ lse, SplitRow* __restrict__ rows, float* __restrict__ part_o,
    float2* __restrict__ part_ml) {
  constexpr int TW = kDecWarps / HC, SU = 2 * TW;  // warps that share a head, units of a step
  constexpr int CT = D / 8;           // channels of a lane's V column
  using X = Tile<D>;
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages];
  __shared__ int abort_flag;
  __shared__ unsigned int est[2];
  DeviceStatus* st = reinterpret_cast<DeviceStatus*>(est);  // the CTA's own (an error touches its first two words)
  __shared__ float red_m[kDecWarps][8], red_l[kDecWarps][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H_kv = pool.H_kv, H_q = H_kv * gs;
  const int stage = stage_bytes(D, TW, H_kv);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int i) { return bar0 + 8u * i; };                  // TMA -> consumers
  auto empty = [&](int i) { return bar0 + 8u * (kMaxStages + i); };  // consumers (8 warps) -> TMA
  float(*red_o)[8][D] = reinterpret_cast<float(*)[8][D]>(sm + stages * stage);  // TW > 1 alone
  griddep_launch_dependents();  // the combine may be scheduled; it waits for this grid's end
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), kDecWarps);
    }
    fence_mbar_init();
    abort_flag = 0;
    est[0] = est[1] = 0u;
  }
  volatile int* abort = &abort_flag;
  Segments sg;
  sg.ctx_len = ctx_len;
  sg.cap = cap;
  sg.n_hb = (H_kv + HC - 1) / HC;
  {
    const FlatSplit fs = flat_split<HC>(ctx_len, B, cap, sg.n_hb);
    sg.f = blockIdx.x * fs.quota;
    sg.f1 = min(fs.total, sg.f + fs.quota);
    sg.before = fs.before;
    sg.seq = fs.seq;
    if (threadIdx.x == 0) {
      SplitRow row = {-1, 0, 0, 0, 0, 0u, 0u, 0};
      if (sg.next() && sg.u0 > 0) {  // the run begins inside a row
        const int64_t r0 = sg.f - sg.u0, c = blockIdx.x;
        const int c0 = (int)(r0 / fs.quota);
        if (c0 == c - 1) {
          row.seq = sg.seq;
          row.hb = sg.hb;
          row.c0 = c0;
          row.c1 = (int)((r0 + sg.T - 1) / fs.quota);
          row.part0 = r0 == c0 * fs.quota ? 0 : 1;
        }
      }
      rows[blockIdx.x] = row;
    }
  }
  const float kInf = __int_as_float(0x7f800000);
  constexpr int kScales = 32 * X::BYTES;  // offset of the scales in a stage
  const int sc_unit = kUnit * H_kv * kGroups, sc_half = sc_unit / 2;

  const int r = lane >> 2, c = lane & 3;
  const int hl = warp % HC, tl = warp / HC;
  const float sl2 = scale * (1.4426950408889634f * kSubUnscale), lazy = kLazy / sl2;  // of scores as they come out
  // this lane's places in its tile: K rows perm(r) (and 8 more), V tokens perm(2c) and perm(2c + 1) (and 8 more)
  const int tile = (2 * tl * HC + hl) * X::BYTES;  // of the warp's first unit; the second one's is HC tiles on
  const int k_at = tile + X::at(X::perm(r), (X::CB / 4) * c);
  const int v_at0 = 16 * X::BYTES + tile + X::at(X::perm(2 * c), (X::CB / 8) * r);
  const int v_at1 = 16 * X::BYTES + tile + X::at(X::perm(2 * c + 1), (X::CB / 8) * r);
  // the ring's next stage and the parity of its use
  int slot = 0;
  uint32_t phase = 0, at = smem_u32(sm);
  const int ahead = stages - 1;  // steps fetched ahead
  bool ok = true;
  uint32_t fetched = 0;  // stages that this warp has filled, and from bit 16 on the parity of the last time
  for (int part = 0; sg.next(); sg.done()) {
    if (sg.bad && threadIdx.x == 0) raise_error(st, kErrBadIndex, 8u);
    const int steps = sg.len > 0 ? (int)((sg.u1 - sg.u0 + SU - 1) / SU) : 0;
    // step i into the stage `off` past `slot`
    auto fetch = [&](int i, int off) {
      int fs = slot + off;
      uint32_t fp = phase;
      if (fs >= stages) fs -= stages, fp ^= 1u;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(empty(fs), fp ^ 1u, abort, st, 0xE01)))) return;
      const int64_t u = sg.u0 + (int64_t)i * SU + lane;  // lanes 0 .. SU - 1: a unit each
      const int n = (int)min((int64_t)SU, sg.u1 - u + lane);
      if (lane == 0) mbar_arrive_expect_tx(full(fs), (uint32_t)(n * (2 * HC * X::BYTES + 2 * sc_unit)));
      fetched = (fetched & ~(0x10000u << fs)) | 1u << fs | fp << (16 + fs);
      __syncwarp();
      if (lane < n) {
        const uint32_t upp = (uint32_t)map.page / kUnit, lp = (uint32_t)u / upp;
        const int in_page = (int)((uint32_t)u - lp * upp) * kUnit;
        int32_t pp = __ldg(map.table + (int64_t)sg.seq * map.max_pages + lp);
        if (pp < 0 || (int64_t)pp >= map.n_pages) {
          raise_error(st, kErrBadIndex, 3u);
          pp = 0;
        }
        const uint32_t to = smem_u32(sm) + fs * stage;
        // tiles in (unit, head) order; a page holds whole units
        tma_load_4d(to + lane * HC * X::BYTES, &tm_k, 0, in_page, sg.hb * HC, pp, full(fs));
        tma_load_4d(to + 16 * X::BYTES + lane * HC * X::BYTES, &tm_v, 0, in_page, sg.hb * HC, pp, full(fs));
        const int64_t row = ((int64_t)pp * map.page + in_page) * (H_kv * kGroups);
        bulk_load(to + kScales + lane * sc_unit, pool.k_scales + row, (uint32_t)sc_unit, full(fs));
        bulk_load(to + kScales + (SU + lane) * sc_unit, pool.v_scales + row, (uint32_t)sc_unit, full(fs));
      }
      __syncwarp();
    };
    if (ok && warp < min(ahead, steps)) fetch(warp, warp);
    const int head = sg.hb * HC + hl, seq = sg.seq;
    const int ks_at = kScales + 2 * tl * sc_unit + (X::perm(r) * H_kv + head) * kGroups + c;
    const int vs_at0 = kScales + (SU + 2 * tl) * sc_unit + (X::perm(2 * c) * H_kv + head) * kGroups + (r >> 1);
    const int vs_at1 = kScales + (SU + 2 * tl) * sc_unit + (X::perm(2 * c + 1) * H_kv + head) * kGroups + (r >> 1);
    // the query as B fragments: lane (n = r, c) holds channels (D / 4) c .. of head r of the group
    uint32_t qf[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) qf[i] = 0u;
    const bool on = head < H_kv;
    if (on && r < gs) {
      const uint4* qp = reinterpret_cast<const uint4*>(q + ((int64_t)seq * H_q + head * gs + r) * D + (D / 4) * c);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 y = qp[i];
        qf[4 * i] = y.x, qf[4 * i + 1] = y.y, qf[4 * i + 2] = y.z, qf[4 * i + 3] = y.w;
      }
    }
    // running maximum (raw scores), what a score must exceed to move it, and the maximum in log2 units
    float o[D / 16][4], m[2] = {-kInf, -kInf}, thr[2] = {-kInf, -kInf}, z[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    int units = (int)(sg.u1 - sg.u0) - 2 * tl;            // left from this warp's place in the step on
    int left = (int)(sg.len - (sg.u0 + 2 * tl) * kUnit);  // tokens likewise (lengths are int32)
    for (int i = 0; i < steps; ++i, units -= SU, left -= SU * kUnit) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(full(slot), phase, abort, st, 0xE10));
      if (ok && on && units > 0) {
        // A second unit past the run's end holds whatever lay in the stage: its tokens count as past the length.
        const int seen = units > 1 ? left : min(left, kUnit);
        uint32_t ks2[2][2], vs2[2][2], top = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
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
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if ((ks2[h][e] & 0xFFFFu) == kNaNRaw) ks2[h][e] = 0x7FFF7FFFu;
              if ((vs2[h][e] & 0xFFFFu) == kNaNRaw) vs2[h][e] |= 0x7FFFu;
              if ((vs2[h][e] >> 16) == kNaNRaw) vs2[h][e] |= 0x7FFF0000u;
            }
        }
        // S^T = K q^T
        float s[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          s[h][0] = s[h][1] = s[h][2] = s[h][3] = 0.f;
          uint32_t kw[2][D / 32];
#pragma unroll
          for (int e = 0; e < 2; ++e) lds_words(at + k_at + h * HC * X::BYTES + e * 8 * X::CB, kw[e]);
          const SubScale sc[2] = {sub_scale(ks2[h][0]), sub_scale(ks2[h][1])};
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            const uint4 a = expand8_sub(kw[0][w], sc[0]), b = expand8_sub(kw[1][w], sc[1]);
            const uint32_t a0[4] = {a.x, b.x, a.y, b.y}, a1[4] = {a.z, b.z, a.w, b.w};
            const uint32_t q0[2] = {qf[4 * w], qf[4 * w + 1]}, q1[2] = {qf[4 * w + 2], qf[4 * w + 3]};
            mma_bf16_16816(s[h], a0, q0);
            mma_bf16_16816(s[h], a1, q1);
          }
        }
        if (seen < 2 * kUnit) {  // tokens past the length: no score, and whatever lies there stays out of V
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (X::perm(r) + 16 * h >= seen) s[h][0] = s[h][1] = -kInf;
            if (X::perm(r) + 16 * h + 8 >= seen) s[h][2] = s[h][3] = -kInf;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (X::perm(2 * c) + 16 * h + 8 * e >= seen) vs2[h][e] &= 0xFFFF0000u;
              if (X::perm(2 * c + 1) + 16 * h + 8 * e >= seen) vs2[h][e] &= 0x0000FFFFu;
            }
          }
        }
        const float t0 = fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2]));
        const float t1 = fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3]));
        if (__any_sync(0xffffffffu, t0 > thr[0] || t1 > thr[1])) {
          float n[2] = {t0, t1}, a[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) n[e] = fmaxf(n[e], __shfl_xor_sync(0xffffffffu, n[e], y));
            n[e] = fmaxf(n[e], m[e]);
            const float zn = n[e] == -kInf ? 0.f : n[e] * sl2;  // scores of -inf alone weigh 0
            a[e] = m[e] == -kInf ? 1.f : ex2_approx(z[e] - zn);
            m[e] = n[e];
            z[e] = zn;
            thr[e] = n[e] == -kInf ? -kInf : n[e] + lazy;
            l[e] *= a[e];
          }
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            o[x][0] *= a[0], o[x][2] *= a[0];
            o[x][1] *= a[1], o[x][3] *= a[1];
          }
        }
        uint32_t pb[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p0 = ex2_approx(fmaf(s[h][0], sl2, -z[0])), p1 = ex2_approx(fmaf(s[h][1], sl2, -z[1]));
          const float p2 = ex2_approx(fmaf(s[h][2], sl2, -z[0])), p3 = ex2_approx(fmaf(s[h][3], sl2, -z[1]));
          l[0] += p0 + p2;
          l[1] += p1 + p3;
          // P^T as a B operand (tokens x heads): the 8 x 8 halves transposed across the warp
          pb[h][0] = movmatrix_t(pack_bf16x2(p0, p1));
          pb[h][1] = movmatrix_t(pack_bf16x2(p2, p3));
        }
        // O^T += V^T P^T
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t vw[4][D / 64];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            lds_words(at + h * HC * X::BYTES + ((e & 1) ? v_at1 : v_at0) + (e >> 1) * 8 * X::CB, vw[e]);
          const SubScale sc[2] = {sub_scale(vs2[h][0]), sub_scale(vs2[h][1])};
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
            // halves of the same nibbles of two tokens side by side: even channels from the low halves, odd from the high
            uint32_t ev[2], od[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              ev[e] = __byte_perm(vw[2 * e][w], vw[2 * e + 1][w], 0x5410);
              od[e] = __byte_perm(vw[2 * e][w], vw[2 * e + 1][w], 0x7632);
            }
            const uint4 e0 = expand8_sub(ev[0], sc[0]), e1 = expand8_sub(ev[1], sc[1]);
            const uint4 d0 = expand8_sub(od[0], sc[0]), d1 = expand8_sub(od[1], sc[1]);
            const uint32_t a0[4] = {e0.x, d0.x, e1.x, d1.x}, a1[4] = {e0.y, d0.y, e1.y, d1.y};
            const uint32_t a2[4] = {e0.z, d0.z, e1.z, d1.z}, a3[4] = {e0.w, d0.w, e1.w, d1.w};
            mma_bf16_16816(o[4 * w], a0, pb[h]);
            mma_bf16_16816(o[4 * w + 1], a1, pb[h]);
            mma_bf16_16816(o[4 * w + 2], a2, pb[h]);
            mma_bf16_16816(o[4 * w + 3], a3, pb[h]);
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
    // ---- the segment's result: l over the token rows, then over the head's TW warps (z: the maximum in log2 units)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int y = 4; y < 32; y <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], y);
      m[e] = m[e] == -kInf ? -kInf : z[e];
    }
    if (TW > 1) {
      if (r == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) red_m[warp][2 * c + e] = m[e], red_l[warp][2 * c + e] = l[e];
      }
      __syncthreads();
      float M[2] = {-kInf, -kInf}, w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        for (int y = 0; y < TW; ++y) M[e] = fmaxf(M[e], red_m[y * HC + hl][2 * c + e]);
        w[e] = m[e] == M[e] ? 1.f : ex2_approx(m[e] - M[e]);
        l[e] = 0.f;
        for (int y = 0; y < TW; ++y) {
          const float my = red_m[y * HC + hl][2 * c + e];
          l[e] += red_l[y * HC + hl][2 * c + e] * (my == M[e] ? 1.f : ex2_approx(my - M[e]));
        }
        m[e] = M[e];
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const int ch = CT * r + 8 * (i / 4) + 2 * (i % 4);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          red_o[warp][2 * c + e][ch] = o[i][e] * w[e];
          red_o[warp][2 * c + e][ch + 1] = o[i][2 + e] * w[e];
        }
      }
      __syncthreads();
      if (tl == 0) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int ch = CT * r + 8 * (i / 4) + 2 * (i % 4);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x0 = 0.f, x1 = 0.f;
            for (int y = 0; y < TW; ++y) {
              x0 += red_o[y * HC + hl][2 * c + e][ch];
              x1 += red_o[y * HC + hl][2 * c + e][ch + 1];
            }
            o[i][e] = x0;
            o[i][2 + e] = x1;
          }
        }
      }
      __syncthreads();  // red_* are free again
    }
    if (tl == 0 && on) {
      const bool whole = sg.u0 == 0 && sg.u1 == sg.T;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hh = 2 * c + e;  // head of the group
        if (hh >= gs) continue;
        if (whole) {
          const bool any = l[e] > 0.f || l[e] != l[e];
          const float inv = any ? kSubUnscale / l[e] : 0.f;
          uint32_t* op = reinterpret_cast<uint32_t*>(out + ((int64_t)seq * H_q + head * gs + hh) * D + CT * r);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) op[i] = pack_bf16x2(o[i][e] * inv, o[i][2 + e] * inv);
          if (r == 0 && lse)
            lse[(int64_t)seq * H_q + head * gs + hh] = any ? (m[e] + log2f(l[e])) * 0.69314718055994530942f : -kInf;
        } else {
          const int64_t slot = (((int64_t)blockIdx.x * 2 + part) * HC + hl) * gs + hh;
          float2* po = reinterpret_cast<float2*>(part_o + slot * D + CT * r);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) po[i] = make_float2(o[i][e], o[i][2 + e]);
          if (r == 0) part_ml[slot] = make_float2(m[e], l[e]);
        }
      }
    }
    part = 1;  // the segment that began the CTA's run is its partial 0, a later one partial 1
  }
  if (*abort && lane == 0)  // a wait gave up: let this warp's copies land before the CTA ends
    for (int i = 0; i < stages; ++i)
      if (fetched >> i & 1u) mbar_wait(full(i), fetched >> (16 + i) & 1u, nullptr, st, 0xEF1);
  __syncthreads();
  if (threadIdx.x == 0 && st->flags) {
    rows[blockIdx.x].flags = st->flags;
    rows[blockIdx.x].first_code = st->first_code;
  }
}

// Merges the partials of the rows that CTAs share: a CTA per (row, two heads), 4 warps a head, each with every 4th
// partial.  Row blockIdx.x is that of the blockIdx.x-th record that names one; CTA 0 also sums up the errors.  (Rows
// found by searching the lengths and a CTA a row took 107 us instead of 84 at 48 sequences of 1200 to 12000 tokens.)
template <int D>
__global__ void __launch_bounds__(kCombThreads) kv4_combine_kernel(const SplitRow* __restrict__ rows, int n_cta, int H_kv,
                                                                  int HC, int gs, const float* __restrict__ part_o,
                                                                  const float2* __restrict__ part_ml,
                                                                  uint16_t* __restrict__ out, float* __restrict__ lse,
                                                                  DeviceStatus* st) {
  constexpr int V = D / 32;  // channels of a lane
  __shared__ float acc_s[2][4][D];
  __shared__ float2 l_s[2][4];  // each warp's maximum and sum
  __shared__ SplitRow row_s;
  __shared__ int named[kCombThreads / 32];
  __shared__ unsigned int est[2];
  const bool first = blockIdx.x == 0 && blockIdx.y == 0;
  if (threadIdx.x == 0) row_s.seq = -1, est[0] = est[1] = 0u;
  griddep_wait();  // the records and the partials
  for (int c0 = 0, before = 0; c0 < n_cta; c0 += kCombThreads) {
    const int ct = c0 + threadIdx.x;
    SplitRow row;
    row.seq = -1, row.flags = 0u;
    if (ct < n_cta) {
      const int4* p = reinterpret_cast<const int4*>(rows + ct);
      *reinterpret_cast<int4*>(&row) = p[0];
      *(reinterpret_cast<int4*>(&row) + 1) = p[1];
    }
    const unsigned int has = __ballot_sync(0xffffffffu, row.seq >= 0);
    __syncthreads();  // named is read (and row_s, est begun)
    if ((threadIdx.x & 31) == 0) named[threadIdx.x >> 5] = __popc(has);
    if (first && row.flags) {
      atomicOr(&est[0], row.flags);
      est[1] = row.first_code;  // any of them
    }
    __syncthreads();
    int rank = before + __popc(has & ((1u << (threadIdx.x & 31)) - 1u));
    for (int x = 0; x < kCombThreads / 32; ++x) {
      before += named[x];
      if (x < (int)threadIdx.x >> 5) rank += named[x];
    }
    if (row.seq >= 0 && rank == (int)blockIdx.x) row_s = row;
  }
  __syncthreads();
  if (first && threadIdx.x == 0) {
    st->flags = est[0];
    st->first_code = est[1];
  }
  const SplitRow row = row_s;
  if (row.seq < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp & 3;
  const int h = blockIdx.y * 2 + (warp >> 2);  // head of the block
  const int heads = min(HC * gs, (H_kv - row.hb * HC) * gs);
  const bool on = h < heads;
  const float kInf = __int_as_float(0x7f800000);
  auto slot_of = [&](int ct) { return ((int64_t)ct * 2 + (ct == row.c0 ? row.part0 : 0)) * (HC * gs) + h; };
  float M = -kInf, L = 0.f, acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  if (on) {
    for (int c0 = row.c0 + w; c0 <= row.c1; c0 += 16) {  // four partials of the warp in flight
      float2 ml[4];
      float x[4][V];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int ct = c0 + 4 * u;
        ml[u] = make_float2(-kInf, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) x[u][i] = 0.f;
        if (ct <= row.c1) {
          const int64_t sl = slot_of(ct);
          const float* p = part_o + sl * D + lane * V;
          ml[u] = part_ml[sl];
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
      L *= old;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] *= old;
      M = m;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float wt = ml[u].x == m ? 1.f : ex2_approx(ml[u].x - m);
        L += ml[u].y * wt;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += x[u][i] * wt;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) acc_s[warp >> 2][w][lane * V + i] = acc[i];
    if (lane == 0) l_s[warp >> 2][w] = make_float2(M, L);
  }
  __syncthreads();
  if (!on || w != 0) return;
  float2 ml[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) ml[u] = l_s[warp >> 2][u];
  M = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
  L = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float wt = ml[u].x == M ? 1.f : ex2_approx(ml[u].x - M);
    L += ml[u].y * wt;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += acc_s[warp >> 2][u][lane * V + i] * wt;
  }
  const bool any = L > 0.f || L != L;  // scores of -inf alone weigh nothing: out 0, lse -inf
  const float inv = any ? kSubUnscale / L : 0.f;  // (partial O comes scaled like V's values)
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] *= inv;
  const int64_t hq = (int64_t)row.seq * (H_kv * gs) + row.hb * HC * gs + h;
  uint32_t* op = reinterpret_cast<uint32_t*>(out + hq * D + lane * V);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) op[i] = pack_bf16x2(acc[2 * i], acc[2 * i + 1]);
  if (lane == 0 && lse) lse[hq] = any ? (M + log2f(L)) * 0.69314718055994530942f : -kInf;
}

int decode_ctas() { return 2 * num_sms(); }

template <int D, int HC>
cudaError_t launch_dense_decode_t(const void* q, const Kv4Pool& pool, const CacheMap& map, const int32_t* ctx_len, int B,
                                  int64_t cap, int gs, float scale, void* out, float* lse, SplitRow* rows,
                                  float* part_o, float2* part_ml, DeviceStatus* st, cudaStream_t s) {
  constexpr int TW = kDecWarps / HC, CB = D / 2;
  alignas(64) unsigned char tk[128], tv[128];
  // codes [n_pages][page][H_kv][CB] bytes (as 16-bit words) in the order {row, token, head, page}
  const uint64_t dims[4] = {CB / 2, (uint64_t)pool.page, (uint64_t)pool.H_kv, (uint64_t)pool.n_pages};
  const uint64_t strides[3] = {(uint64_t)pool.H_kv * CB, CB, (uint64_t)pool.page * pool.H_kv * CB};
  const uint32_t box[4] = {CB / 2, kUnit, HC, 1};
  if (!encode_tmap_4d(tk, pool.k_codes, dims, strides, box, CB) || !encode_tmap_4d(tv, pool.v_codes, dims, strides, box, CB))
    return cudaErrorInvalidValue;
  const int stage = stage_bytes(D, TW, pool.H_kv), red = TW > 1 ? kDecWarps * 8 * D * 4 : 0;
  const int fit = (kDecSmem - 1024 - red) / stage, stages = fit > kMaxStages ? kMaxStages : fit;
  const int smem = 1024 + stages * stage + red;
  const int n_cta = decode_ctas();
  auto kern = kv4_dense_decode_kernel<D, HC>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kDecSmem);
  if (e != cudaSuccess) return e;
  kern<<<n_cta, kDecThreads, smem, s>>>(*reinterpret_cast<const CUtensorMap*>(tk), *reinterpret_cast<const CUtensorMap*>(tv),
                                        (const uint16_t*)q, pool, map, ctx_len, B, cap, gs, scale, stages, (uint16_t*)out,
                                        lse, rows, part_o, part_ml);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int64_t most = (int64_t)B * ((pool.H_kv + HC - 1) / HC);  // rows; at most one split a CTA boundary
  cfg.gridDim = dim3((unsigned)(most < n_cta ? most : n_cta), (unsigned)(HC * gs + 1) / 2);
  cfg.blockDim = dim3(kCombThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_combine_kernel<D>, (const SplitRow*)rows, n_cta, pool.H_kv, HC, gs,
                            (const float*)part_o, (const float2*)part_ml, (uint16_t*)out, lse, st);
}

// Heads of a CTA: all of up to 8, so that a token's scales come as one run; for H_kv > 4 always 8 (8 heads,
// 4 sequences of 2^20 tokens: 1303 us with 4 a CTA, 829 with 8; 48 of 1200 to 12000: 128 and 84), for fewer the next power
// of two, the warps left over sharing a head's tokens.
int heads_per_cta(int H_kv) { return H_kv > 4 ? 8 : H_kv > 2 ? 4 : H_kv; }

}  // namespace

// Rounds of a CTA: four CTAs an SM at least before a CTA takes a second round.
static int rows_rounds(int64_t N, int tpp) {
  const int64_t r = N / ((int64_t)4 * num_sms() * kUnroll * tpp);
  return r > kRounds ? kRounds : r < 1 ? 1 : (int)r;
}

cudaError_t launch_kv4_store(const void* k, const void* v, int64_t N, const int32_t* cu, int S, const int32_t* pos0,
                             const int32_t* table, int64_t max_pages, const Kv4Pool& pool, DeviceStatus* st, cudaStream_t s) {
  const RowMap map = row_map(cu, S, pos0, table, max_pages, pool.n_pages, pool.page);
  const int tpp = RowTile(pool.H_kv, pool.d / 8).tpp, R = rows_rounds(N, tpp);
  auto kern = pool.d == 64 ? kv4_store_kernel<64> : kv4_store_kernel<128>;
  kern<<<(unsigned)ceil_div(N, R * kUnroll * tpp), kRowThreads, 0, s>>>((const uint16_t*)k, (const uint16_t*)v, N, R, map,
                                                                       pool, st);
  return cudaGetLastError();
}

cudaError_t launch_kv4_load(const Kv4Pool& pool, int64_t N, const int32_t* cu, int S, const int32_t* pos0,
                            const int32_t* table, int64_t max_pages, void* k, void* v, DeviceStatus* st, cudaStream_t s) {
  const RowMap map = row_map(cu, S, pos0, table, max_pages, pool.n_pages, pool.page);
  const int tpp = RowTile(pool.H_kv, pool.d / 8).tpp, R = rows_rounds(N, tpp);
  auto kern = pool.d == 64 ? kv4_load_kernel<64> : kv4_load_kernel<128>;
  kern<<<(unsigned)ceil_div(N, R * kUnroll * tpp), kRowThreads, 0, s>>>(pool, N, R, map, (uint16_t*)k, (uint16_t*)v, st);
  return cudaGetLastError();
}

// Scratch: a record of each CTA, the partials.
struct DecScratch {
  SplitRow* rows;
  float* part_o;
  float2* part_ml;
};
static size_t carve_dense_decode(int H_kv, int gs, int d, char* base, DecScratch* out) {
  const size_t slots = (size_t)decode_ctas() * 2 * heads_per_cta(H_kv) * gs;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* r = base ? base + off : nullptr;
    off += align_up(bytes, 256);
    return r;
  };
  DecScratch w;
  w.rows = (SplitRow*)take((size_t)decode_ctas() * sizeof(SplitRow));
  w.part_o = (float*)take(slots * d * 4);
  w.part_ml = (float2*)take(slots * 8);
  if (out) *out = w;
  return off;
}

size_t dense_decode_scratch_bytes(int H_kv, int gs, int d) { return carve_dense_decode(H_kv, gs, d, nullptr, nullptr); }

cudaError_t launch_dense_decode(const void* q, const Kv4Pool& pool, const int32_t* table, int64_t max_pages,
                                const int32_t* ctx_len, int B, int H_q, float scale, void* out, float* lse, void* scratch,
                                DeviceStatus* st, cudaStream_t s) {
  const int gs = H_q / pool.H_kv, HC = heads_per_cta(pool.H_kv);
  DecScratch w;
  carve_dense_decode(pool.H_kv, gs, pool.d, (char*)scratch, &w);
  CacheMap map;
  map.table = table;
  map.max_pages = max_pages;
  map.n_pages = pool.n_pages;
  map.page = pool.page;
  const int64_t cap = max_pages * pool.page;
#define MSA_DD(D, H) \
  launch_dense_decode_t<D, H>(q, pool, map, ctx_len, B, cap, gs, scale, out, lse, w.rows, w.part_o, w.part_ml, st, s)
  if (pool.d == 64) return HC == 8 ? MSA_DD(64, 8) : HC == 4 ? MSA_DD(64, 4) : HC == 2 ? MSA_DD(64, 2) : MSA_DD(64, 1);
  return HC == 8 ? MSA_DD(128, 8) : HC == 4 ? MSA_DD(128, 4) : HC == 2 ? MSA_DD(128, 2) : MSA_DD(128, 1);
#undef MSA_DD
}

}  // namespace msa
