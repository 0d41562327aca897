// Rows of K and V into and out of a 4-bit paged cache, and dense decode over it.
#include <math.h>

#include "msa_kv4.cuh"

namespace msa {

namespace {

using namespace kv4;

constexpr int kRowThreads = 256;

// Where packed row i goes: the pool row of its sequence's token, or -1 (past the last sequence, or bad: flagged).
struct RowMap {
  const int32_t* cu;    // [S + 1]
  const int32_t* pos0;  // [S] token position of each sequence's first row
  const int32_t* table;
  int64_t max_pages, n_pages;
  int S, page;

  __device__ __forceinline__ int64_t row(int64_t i, DeviceStatus* st) const {
    if (i < cu[0] || i >= cu[S]) return -1;
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
    return (int64_t)pp * page + (t - lp * page);
  }
};

// One warp per packed row (token): 8 channels of a head row a lane, K's head rows then V's.  A group is 4
// (d = 128) or 2 (d = 64) lanes, whose shared maximum gives its scale.
template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_store_kernel(const uint16_t* __restrict__ k,
                                                                const uint16_t* __restrict__ v, int64_t N, RowMap map,
                                                                Kv4Pool pool, DeviceStatus* st) {
  constexpr int LPR = D / 8, LPG = LPR / kGroups;
  const int lane = threadIdx.x & 31;
  const int64_t stride = (int64_t)gridDim.x * (kRowThreads / 32);
  for (int64_t i = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); i < N; i += stride) {
    const int64_t row = map.row(i, lane == 0 ? st : nullptr);
    if (row < 0) continue;
    const int tasks = pool.H_kv * LPR;
#pragma unroll 1
    for (int c0 = 0; c0 < 2 * tasks; c0 += 32) {
      const int c = c0 + lane;
      const bool in = c < 2 * tasks, is_v = c >= tasks;
      const int e = is_v ? c - tasks : c;  // 8-channel piece of the token's K or V
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (in) x = ldg_stream_16((is_v ? v : k) + (i * tasks + e) * 8);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t mx = 0u;  // largest |x| as bf16 bits: magnitudes order as integers, NaN and infinity on top
#pragma unroll
      for (int j = 0; j < 4; ++j) mx = max(mx, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
#pragma unroll
      for (int o = 1; o < LPG; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const bool bad = mx >= 0x7F80u;
      const uint32_t sb = bad ? kScaleNaN : scale_of(mx);
      const float inv = bad ? 0.f : 1.0f / scale_f32(sb);
      uint32_t code = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // channels 2j, 2j + 1 -> nibbles j, j + 4
        code |= (bad ? 8u : code_of(bf16_lo(w[j]), inv)) << (4 * j);
        code |= (bad ? 8u : code_of(bf16_hi(w[j]), inv)) << (4 * j + 16);
      }
      if (in) {
        uint8_t* codes = is_v ? pool.v_codes : pool.k_codes;
        uint8_t* scales = is_v ? pool.v_scales : pool.k_scales;
        reinterpret_cast<uint32_t*>(codes)[row * tasks + e] = code;
        if (lane % LPG == 0) scales[row * (pool.H_kv * kGroups) + e / LPG] = (uint8_t)sb;
      }
    }
  }
}

// The same rows back as exact bf16 values; zeros where the row map has no place.
template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_load_kernel(Kv4Pool pool, int64_t N, RowMap map,
                                                               uint16_t* __restrict__ k, uint16_t* __restrict__ v,
                                                               DeviceStatus* st) {
  constexpr int LPR = D / 8, LPG = LPR / kGroups;
  const int lane = threadIdx.x & 31;
  const int64_t stride = (int64_t)gridDim.x * (kRowThreads / 32);
  for (int64_t i = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); i < N; i += stride) {
    if (i >= map.cu[map.S] || i < map.cu[0]) continue;  // rows of no sequence stay as they were
    const int64_t row = map.row(i, lane == 0 ? st : nullptr);
    const int tasks = pool.H_kv * LPR;
    for (int c = lane; c < 2 * tasks; c += 32) {
      const bool is_v = c >= tasks;
      const int e = is_v ? c - tasks : c;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (row >= 0) {
        const uint8_t* codes = is_v ? pool.v_codes : pool.k_codes;
        const uint8_t* scales = is_v ? pool.v_scales : pool.k_scales;
        const uint32_t s = scale_bf16(scales[row * (pool.H_kv * kGroups) + e / LPG]), s2 = s | (s << 16);
        x = expand8(reinterpret_cast<const uint32_t*>(codes)[row * tasks + e], s2, scale_bias(s2));
      }
      *reinterpret_cast<uint4*>((is_v ? v : k) + (i * tasks + e) * 8) = x;
    }
  }
}

// ---------------------------------------------------------------- dense decode
// One query token per sequence against its whole cache.  The caches are read
// as one flat list of 16-token units, ordered by (sequence, head block, unit),
// a head block being HC heads of the 8 warps' (HC = 8, 4, 2 or 1, whichever
// divides H_kv); every CTA takes an equal run of it, whatever the lengths are.
// A run that covers a (sequence, head block) row whole writes its output; the
// others leave (O, max, sum) partials, at most two a CTA, for the combine.
constexpr int kUnit = 16;
constexpr int kDecThreads = 256, kDecWarps = 8;
constexpr float kLazy = 8.0f;  // log2 units a row maximum may grow before O is rescaled

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Units of sequence s (at least one, so that an empty sequence's output is written); a length outside
// [0, cap] counts as 0.
__device__ __forceinline__ int64_t units_of(int32_t len, int64_t cap) {
  return len <= 0 || (int64_t)len > cap ? 1 : ((int64_t)len + kUnit - 1) / kUnit;
}

// Units of a CTA's run: a multiple of the warps that share a head, so that none of them starts idle.
__device__ __forceinline__ int64_t quota_of(int64_t total, int n_cta, int tw) {
  return ((total + n_cta - 1) / n_cta + tw - 1) / tw * tw;
}

// The split of the flat unit list, worked out by every CTA from the lengths.
struct FlatSplit {
  int64_t total;   // units over all sequences and head blocks
  int64_t quota;   // units a CTA takes
  int64_t before;  // units (times head blocks) before sequence `seq`
  int seq;         // the sequence that holds unit `want` (B if none)
};

// Block-wide sums over the sequences; want(total, quota) names the unit to look for.
template <int HC, typename F>
__device__ __forceinline__ FlatSplit flat_split(const int32_t* ctx_len, int B, int64_t cap, int n_hb, int n_cta, F want) {
  __shared__ int64_t part[kDecWarps], found_before;
  __shared__ int found_seq;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t sum = 0;
  for (int s = tid; s < B; s += kDecThreads) sum += units_of(ctx_len[s], cap);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) part[warp] = sum;
  if (tid == 0) found_seq = B;
  __syncthreads();
  FlatSplit f;
  f.total = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) f.total += part[w];
  f.total *= n_hb;
  f.quota = quota_of(f.total, n_cta, kDecWarps / HC);
  const int64_t at = want(f.total, f.quota);
  int64_t base = 0;
  for (int s0 = 0; s0 < B; s0 += kDecThreads) {
    const int s = s0 + tid;
    const int64_t n = s < B ? units_of(ctx_len[s], cap) : 0;
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    __syncthreads();  // part of the step before is no longer read
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int64_t off = base;
    for (int w = 0; w < kDecWarps; ++w) {
      if (w < warp) off += part[w];
      base += part[w];
    }
    const int64_t lo = (off + incl - n) * n_hb, hi = (off + incl) * n_hb;
    if (s < B && lo <= at && at < hi) {
      found_seq = s;
      found_before = lo;
    }
    if (base * n_hb > at) break;  // uniform
  }
  __syncthreads();
  f.seq = found_seq;
  f.before = found_before;
  return f;
}

// A warp's units pass through a ring of kStages in shared memory (cp.async), so that the bytes in flight do not
// depend on registers: 2 CTAs x 8 warps x 5 units of 2176 bytes (d = 128) an SM.
constexpr int kStages = 6;
template <int D>
struct Ring {
  static constexpr int CODES = kUnit * D / 2;                 // bytes of a unit's codes of one head
  static constexpr int K = 0, V = CODES, KS = 2 * CODES, VS = KS + kUnit * kGroups;
  static constexpr int STAGE = VS + kUnit * kGroups;
  static constexpr int WARP = kStages * STAGE;
  static constexpr int SMEM = kDecWarps * WARP;
};
static_assert(Ring<64>::SMEM >= kDecWarps * 8 * 64 * 4 && Ring<128>::SMEM >= kDecWarps * 8 * 128 * 4, "red_o fits over the ring");

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_16s(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}

// Where token t's V codes sit in a unit: a lane column c reads tokens 2c, 2c + 1, 2c + 8, 2c + 9, so the four
// columns' tokens lie side by side, and (d = 128) every other pair has its 32-byte halves exchanged: 16 lanes'
// 8-byte reads then fall in distinct banks.
__device__ __forceinline__ int v_slot(int t) { return ((t >> 1) & 3) + 4 * (t & 1) + 8 * (t >> 3); }
template <int D>
__device__ __forceinline__ int v_flip(int slot) { return D == 128 ? 32 * ((slot >> 1) & 1) : 0; }

template <int D, int HC>
__global__ void __launch_bounds__(kDecThreads, 2) kv4_dense_decode_kernel(const uint16_t* __restrict__ q, Kv4Pool pool,
                                                                       CacheMap map, const int32_t* __restrict__ ctx_len,
                                                                       int B, int64_t cap, int gs, float scale,
                                                                       uint16_t* __restrict__ out, float* __restrict__ lse,
                                                                       float* __restrict__ part_o,
                                                                       float2* __restrict__ part_ml, DeviceStatus* st) {
  constexpr int TW = kDecWarps / HC;  // warps that share a head, every TW-th unit each
  constexpr int CB = D / 2;           // bytes of a head row's codes
  constexpr int CT = D / 8;           // channels of a lane's V column
  using R = Ring<D>;
  extern __shared__ __align__(16) uint8_t ring[];
  float(*red_o)[8][D] = reinterpret_cast<float(*)[8][D]>(ring);  // over the ring, between segments
  __shared__ float red_m[kDecWarps][8], red_l[kDecWarps][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int hl = warp % HC, tl = warp / HC;
  const int H_kv = pool.H_kv, n_hb = H_kv / HC, H_q = H_kv * gs;
  const float kInf = __int_as_float(0x7f800000);
  const int64_t cta = blockIdx.x;
  const FlatSplit fs = flat_split<HC>(ctx_len, B, cap, n_hb, gridDim.x, [&](int64_t, int64_t quota) { return cta * quota; });
  int64_t f = cta * fs.quota;
  const int64_t f1 = min(fs.total, f + fs.quota);
  if (f >= f1) return;
  int seq = fs.seq;
  int64_t before = fs.before;
  const float sl2 = scale * 1.4426950408889634f;
  for (int part = 0; f < f1;) {
    const int32_t len_raw = ctx_len[seq];
    const bool bad = len_raw < 0 || (int64_t)len_raw > cap;
    if (bad && threadIdx.x == 0) raise_error(st, kErrBadIndex, 8u);
    const int64_t len = bad ? 0 : len_raw;
    const int64_t T = units_of(len_raw, cap);
    const int hb = (int)((f - before) / T);
    const int64_t r0 = before + hb * T;
    const int64_t u0 = f - r0, u1 = min(f1 - r0, T);  // this segment's units of the row
    const int head = hb * HC + hl;
    // the query as B fragments: lane (n = r, c) holds channels (D / 4) c .. of head r of the group
    uint32_t qf[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) qf[i] = 0u;
    if (r < gs) {
      const uint4* qp = reinterpret_cast<const uint4*>(q + ((int64_t)seq * H_q + head * gs + r) * D + (D / 4) * c);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 x = qp[i];
        qf[4 * i] = x.x, qf[4 * i + 1] = x.y, qf[4 * i + 2] = x.z, qf[4 * i + 3] = x.w;
      }
    }
    float o[D / 16][4], m[2] = {-kInf, -kInf}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    if (len > 0) {
      // this warp's units u0 + tl + i TW: n of them
      const int n = u1 - u0 > tl ? (int)((u1 - u0 - tl + TW - 1) / TW) : 0;
      const uint32_t my_ring = smem_u32(ring) + warp * R::WARP;
      // the page of the next unit to fetch; 32 table entries at a time sit in the lanes
      const int upp = map.page / kUnit;
      int64_t lp = (u0 + tl) / upp, id_base = lp - 32;
      int in_page = (int)((u0 + tl) - lp * upp), ids = 0;
      uint32_t fetch_at = my_ring;
      constexpr int PIECES = D / 32;  // 16-byte pieces of a head row
      auto fetch = [&](int i) {
        if (i < n) {
          if (lp - id_base >= 32) {
            id_base = lp;
            ids = lp + lane < map.max_pages ? __ldg(map.table + (int64_t)seq * map.max_pages + lp + lane) : 0;
          }
          int32_t pp = __shfl_sync(0xffffffffu, ids, (int)(lp - id_base));
          if (pp < 0 || (int64_t)pp >= map.n_pages) {
            if (lane == 0) raise_error(st, kErrBadIndex, 3u);
            pp = 0;
          }
          const int64_t hrow = ((int64_t)pp * map.page + in_page * kUnit) * H_kv + head;
          const uint8_t* ks = pool.k_codes + hrow * CB;
          const uint8_t* vs = pool.v_codes + hrow * CB;
#pragma unroll
          for (int x = 0; x < PIECES / 2; ++x) {
            const int t = (lane + 32 * x) / PIECES, piece = lane % PIECES, slot = v_slot(t);
            cp_async_16s(fetch_at + R::K + t * CB + piece * 16, ks + t * (H_kv * CB) + piece * 16);
            cp_async_16s(fetch_at + R::V + slot * CB + ((piece * 16) ^ v_flip<D>(slot)), vs + t * (H_kv * CB) + piece * 16);
          }
          const int t = lane & 15;
          cp_async_4(fetch_at + R::KS + lane * 4, (lane < 16 ? pool.k_scales : pool.v_scales) + (hrow + t * H_kv) * kGroups);
          in_page += TW;
          while (in_page >= upp) in_page -= upp, ++lp;
        }
        fetch_at = fetch_at + R::STAGE == my_ring + R::WARP ? my_ring : fetch_at + R::STAGE;
        cp_async_commit();
      };
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) fetch(i);
      const uint8_t* at = ring + warp * R::WARP;
      for (int i = 0; i < n; ++i) {
        __syncwarp();  // every lane has read the stage that is now filled again
        fetch(i + kStages - 1);
        cp_async_wait<kStages - 1>();
        __syncwarp();
        const int64_t tok = (u0 + tl + (int64_t)i * TW) * kUnit;
        const bool tail = tok + kUnit > len;
        // S^T = K q^T: token rows r and r + 8, the D / 4 channels (one group) 
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        {
          uint32_t kw[2][D / 32], s2[2], b2[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint8_t* kp = at + R::K + (r + 8 * e) * CB + (CB / 4) * c;
            if constexpr (D == 128) {
              const uint4 x = *reinterpret_cast<const uint4*>(kp);
              kw[e][0] = x.x, kw[e][1] = x.y, kw[e][2] = x.z, kw[e][3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(kp);
              kw[e][0] = x.x, kw[e][1] = x.y;
            }
            const uint32_t sb = scale_bf16(at[R::KS + (r + 8 * e) * kGroups + c]);
            s2[e] = sb | (sb << 16);
            b2[e] = scale_bias(s2[e]);
          }
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint4 x = expand8(kw[0][i], s2[0], b2[0]), y = expand8(kw[1][i], s2[1], b2[1]);
            const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
            const uint32_t q0[2] = {qf[4 * i], qf[4 * i + 1]}, q1[2] = {qf[4 * i + 2], qf[4 * i + 3]};
            mma_bf16_16816(s, a0, q0);
            mma_bf16_16816(s, a1, q1);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] *= sl2;
        if (tail) {
          if (tok + r >= len) s[0] = s[1] = -kInf;
          if (tok + r + 8 >= len) s[2] = s[3] = -kInf;
        }
        const float t0 = fmaxf(s[0], s[2]), t1 = fmaxf(s[1], s[3]);
        if (__any_sync(0xffffffffu, t0 > m[0] + kLazy || t1 > m[1] + kLazy)) {
          float n0 = t0, n1 = t1;
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) {
            n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, x));
            n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, x));
          }
          n0 = fmaxf(n0, m[0]);
          n1 = fmaxf(n1, m[1]);
          const float a0 = m[0] == n0 ? 1.f : ex2(m[0] - n0), a1 = m[1] == n1 ? 1.f : ex2(m[1] - n1);
          m[0] = n0;
          m[1] = n1;
          l[0] *= a0;
          l[1] *= a1;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[i][0] *= a0, o[i][2] *= a0;
            o[i][1] *= a1, o[i][3] *= a1;
          }
        }
        const float z0 = m[0] == -kInf ? 0.f : m[0], z1 = m[1] == -kInf ? 0.f : m[1];
        const float p0 = ex2(s[0] - z0), p1 = ex2(s[1] - z1), p2 = ex2(s[2] - z0), p3 = ex2(s[3] - z1);
        l[0] += p0 + p2;
        l[1] += p1 + p3;
        // P^T as a B operand (tokens x heads): the 8 x 8 halves transposed across the warp
        const uint32_t pb[2] = {movmatrix_t(pack_bf16x2(p0, p1)), movmatrix_t(pack_bf16x2(p2, p3))};
        // O^T += V^T P^T: channels CT r .. of tokens 2c, 2c + 1, 2c + 8, 2c + 9
        uint32_t vw[4][D / 64], vs2[2], vb2[2];
        uint32_t sc[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = 2 * c + (e & 1) + 8 * (e >> 1), slot = c + 4 * (e & 1) + 8 * (e >> 1);
          const uint8_t* vp = at + R::V + slot * CB + (((CB / 8) * r) ^ v_flip<D>(c));
          if constexpr (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(vp);
            vw[e][0] = x.x, vw[e][1] = x.y;
          } else {
            vw[e][0] = *reinterpret_cast<const uint32_t*>(vp);
          }
          sc[e] = scale_bf16(at[R::VS + t * kGroups + (r >> 1)]);
          if (tail && tok + t >= len) sc[e] = 0u;  // weight 0 times whatever lies there stays 0
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          vs2[e] = sc[2 * e] | (sc[2 * e + 1] << 16);
          vb2[e] = scale_bias(vs2[e]);
        }
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          // halves of the same nibbles of two tokens side by side: even channels from the low halves, odd from the high
          uint32_t ev[2], od[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ev[e] = __byte_perm(vw[2 * e][i], vw[2 * e + 1][i], 0x5410);
            od[e] = __byte_perm(vw[2 * e][i], vw[2 * e + 1][i], 0x7632);
          }
          const uint4 e0 = expand8(ev[0], vs2[0], vb2[0]), e1 = expand8(ev[1], vs2[1], vb2[1]);
          const uint4 d0 = expand8(od[0], vs2[0], vb2[0]), d1 = expand8(od[1], vs2[1], vb2[1]);
          const uint32_t a0[4] = {e0.x, d0.x, e1.x, d1.x}, a1[4] = {e0.y, d0.y, e1.y, d1.y};
          const uint32_t a2[4] = {e0.z, d0.z, e1.z, d1.z}, a3[4] = {e0.w, d0.w, e1.w, d1.w};
          mma_bf16_16816(o[4 * i], a0, pb);
          mma_bf16_16816(o[4 * i + 1], a1, pb);
          mma_bf16_16816(o[4 * i + 2], a2, pb);
          mma_bf16_16816(o[4 * i + 3], a3, pb);
        }
        at = at + R::STAGE == ring + warp * R::WARP + R::WARP ? ring + warp * R::WARP : at + R::STAGE;
      }
      cp_async_wait<0>();
    }
    // ---- the segment's result: l over the token rows, then over the head's TW warps
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], x);
    if (TW > 1) {
      if (r == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) red_m[warp][2 * c + e] = m[e], red_l[warp][2 * c + e] = l[e];
      }
      __syncthreads();
      float M[2] = {-kInf, -kInf}, w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        for (int x = 0; x < TW; ++x) M[e] = fmaxf(M[e], red_m[x * HC + hl][2 * c + e]);
        w[e] = m[e] == M[e] ? 1.f : ex2(m[e] - M[e]);
        l[e] = 0.f;
        for (int x = 0; x < TW; ++x) {
          const float mx = red_m[x * HC + hl][2 * c + e];
          l[e] += red_l[x * HC + hl][2 * c + e] * (mx == M[e] ? 1.f : ex2(mx - M[e]));
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
            for (int x = 0; x < TW; ++x) {
              x0 += red_o[x * HC + hl][2 * c + e][ch];
              x1 += red_o[x * HC + hl][2 * c + e][ch + 1];
            }
            o[i][e] = x0;
            o[i][2 + e] = x1;
          }
        }
      }
      __syncthreads();  // the ring and red_* are free again
    }
    if (tl == 0) {
      const bool whole = u0 == 0 && u1 == T;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hh = 2 * c + e;  // head of the group
        if (hh >= gs) continue;
        if (whole) {
          const float inv = l[e] > 0.f || l[e] != l[e] ? 1.f / l[e] : 0.f;
          uint32_t* op = reinterpret_cast<uint32_t*>(out + ((int64_t)seq * H_q + head * gs + hh) * D + CT * r);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) op[i] = pack_bf16x2(o[i][e] * inv, o[i][2 + e] * inv);
          if (r == 0 && lse)
            lse[(int64_t)seq * H_q + head * gs + hh] =
                l[e] > 0.f || l[e] != l[e] ? (m[e] + log2f(l[e])) * 0.69314718055994530942f : -kInf;
        } else {
          const int64_t slot = ((cta * 2 + part) * HC + hl) * gs + hh;
          float2* po = reinterpret_cast<float2*>(part_o + slot * D + CT * r);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) po[i] = make_float2(o[i][e], o[i][2 + e]);
          if (r == 0) part_ml[slot] = make_float2(m[e], l[e]);
        }
      }
    }
    // ---- the next row of this CTA's run; a segment that began the CTA's run is partial 0, a later one partial 1
    part = 1;
    f = r0 + u1;
    if (f >= before + n_hb * T) {
      before += n_hb * T;
      ++seq;
    }
  }
}

// One CTA per (sequence, head block) row: merges the partials of the CTAs that share it.
template <int D>
__global__ void __launch_bounds__(kDecThreads) kv4_combine_kernel(const int32_t* __restrict__ ctx_len, int B, int64_t cap,
                                                                  int H_kv, int HC, int gs, int n_cta,
                                                                  const float* __restrict__ part_o,
                                                                  const float2* __restrict__ part_ml,
                                                                  uint16_t* __restrict__ out, float* __restrict__ lse) {
  const int n_hb = H_kv / HC, seq = blockIdx.x / n_hb, hb = blockIdx.x % n_hb;
  const int tid = threadIdx.x;
  int64_t total = 0, before = 0;
  __shared__ int64_t sums[2][kDecWarps];
  for (int s = tid; s < B; s += kDecThreads) {
    const int64_t n = units_of(ctx_len[s], cap);
    total += n;
    if (s < seq) before += n;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if ((tid & 31) == 0) sums[0][tid >> 5] = total, sums[1][tid >> 5] = before;
  __syncthreads();
  total = before = 0;
  for (int w = 0; w < kDecWarps; ++w) total += sums[0][w], before += sums[1][w];
  total *= n_hb;
  const int64_t quota = quota_of(total, n_cta, kDecWarps / HC);
  const int64_t T = units_of(ctx_len[seq], cap);
  const int64_t r0 = before * n_hb + hb * T, r1 = r0 + T;
  const int c0 = (int)(r0 / quota), c1 = (int)((r1 - 1) / quota);
  if (c0 == c1) return;  // one CTA held the row whole
  const int heads = HC * gs, H_q = H_kv * gs;
  auto slot_of = [&](int ct, int h) {  // a row that holds the CTA's first unit is its partial 0
    return ((int64_t)ct * 2 + (r0 <= ct * quota ? 0 : 1)) * heads + h;
  };
  for (int e = tid; e < heads * (D / 4); e += kDecThreads) {
    const int h = e / (D / 4), ch = 4 * (e % (D / 4));
    float M = __int_as_float(0xff800000);
    for (int ct = c0; ct <= c1; ++ct) M = fmaxf(M, part_ml[slot_of(ct, h)].x);
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int ct = c0; ct <= c1; ++ct) {
      const int64_t sl = slot_of(ct, h);
      const float2 ml = part_ml[sl];
      const float w = ml.x == M ? 1.f : ex2(ml.x - M);
      const float4 x = *reinterpret_cast<const float4*>(part_o + sl * D + ch);
      L += ml.y * w;
      acc.x += x.x * w, acc.y += x.y * w, acc.z += x.z * w, acc.w += x.w * w;
    }
    const bool any = L > 0.f || L != L;  // scores of -inf alone weigh nothing: out 0, lse -inf
    const float inv = any ? 1.f / L : 0.f;
    const int64_t hq = (int64_t)seq * H_q + hb * heads + h;
    *reinterpret_cast<uint2*>(out + hq * D + ch) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (ch == 0 && lse) lse[hq] = any ? (M + log2f(L)) * 0.69314718055994530942f : __int_as_float(0xff800000);
  }
}

RowMap row_map(const Kv4Pool& pool, const int32_t* cu, int S, const int32_t* pos0, const int32_t* table, int64_t max_pages) {
  RowMap m;
  m.cu = cu;
  m.pos0 = pos0;
  m.table = table;
  m.max_pages = max_pages;
  m.n_pages = pool.n_pages;
  m.S = S;
  m.page = pool.page;
  return m;
}

unsigned row_grid(int64_t N) {
  const int64_t want = ceil_div(N, kRowThreads / 32), most = (int64_t)num_sms() * 8;
  return (unsigned)(want < most ? want : most);
}

int decode_ctas() { return 2 * num_sms(); }

template <int D, int HC>
cudaError_t launch_dense_decode_t(const void* q, const Kv4Pool& pool, const CacheMap& map, const int32_t* ctx_len, int B,
                                  int64_t cap, int gs, float scale, void* out, float* lse, float* part_o, float2* part_ml,
                                  DeviceStatus* st, cudaStream_t s) {
  const int n_cta = decode_ctas();
  auto kern = kv4_dense_decode_kernel<D, HC>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<D>::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<n_cta, kDecThreads, Ring<D>::SMEM, s>>>((const uint16_t*)q, pool, map, ctx_len, B, cap, gs, scale, (uint16_t*)out,
                                                 lse, part_o, part_ml, st);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  kv4_combine_kernel<D><<<(unsigned)(B * (pool.H_kv / HC)), kDecThreads, 0, s>>>(ctx_len, B, cap, pool.H_kv, HC, gs, n_cta,
                                                                                 part_o, part_ml, (uint16_t*)out, lse);
  return cudaGetLastError();
}

int heads_per_cta(int H_kv) { return H_kv % 8 == 0 ? 8 : H_kv % 4 == 0 ? 4 : H_kv % 2 == 0 ? 2 : 1; }

}  // namespace

cudaError_t launch_kv4_store(const void* k, const void* v, int64_t N, const int32_t* cu, int S, const int32_t* pos0,
                             const int32_t* table, int64_t max_pages, const Kv4Pool& pool, DeviceStatus* st, cudaStream_t s) {
  const RowMap map = row_map(pool, cu, S, pos0, table, max_pages);
  if (pool.d == 64)
    kv4_store_kernel<64><<<row_grid(N), kRowThreads, 0, s>>>((const uint16_t*)k, (const uint16_t*)v, N, map, pool, st);
  else
    kv4_store_kernel<128><<<row_grid(N), kRowThreads, 0, s>>>((const uint16_t*)k, (const uint16_t*)v, N, map, pool, st);
  return cudaGetLastError();
}

cudaError_t launch_kv4_load(const Kv4Pool& pool, int64_t N, const int32_t* cu, int S, const int32_t* pos0,
                            const int32_t* table, int64_t max_pages, void* k, void* v, DeviceStatus* st, cudaStream_t s) {
  const RowMap map = row_map(pool, cu, S, pos0, table, max_pages);
  if (pool.d == 64)
    kv4_load_kernel<64><<<row_grid(N), kRowThreads, 0, s>>>(pool, N, map, (uint16_t*)k, (uint16_t*)v, st);
  else
    kv4_load_kernel<128><<<row_grid(N), kRowThreads, 0, s>>>(pool, N, map, (uint16_t*)k, (uint16_t*)v, st);
  return cudaGetLastError();
}

size_t dense_decode_scratch_bytes(int H_kv, int gs, int d) {
  const size_t slots = (size_t)decode_ctas() * 2 * heads_per_cta(H_kv) * gs;
  return align_up(slots * d * 4, 256) + align_up(slots * 8, 256);
}

cudaError_t launch_dense_decode(const void* q, const Kv4Pool& pool, const int32_t* table, int64_t max_pages,
                                const int32_t* ctx_len, int B, int H_q, float scale, void* out, float* lse, void* scratch,
                                DeviceStatus* st, cudaStream_t s) {
  const int gs = H_q / pool.H_kv, HC = heads_per_cta(pool.H_kv);
  const size_t slots = (size_t)decode_ctas() * 2 * HC * gs;
  float* po = (float*)scratch;
  float2* ml = (float2*)((char*)scratch + align_up(slots * pool.d * 4, 256));
  CacheMap map;
  map.table = table;
  map.max_pages = max_pages;
  map.n_pages = pool.n_pages;
  map.page = pool.page;
  const int64_t cap = max_pages * pool.page;
#define MSA_DD(D, H) launch_dense_decode_t<D, H>(q, pool, map, ctx_len, B, cap, gs, scale, out, lse, po, ml, st, s)
  if (pool.d == 64) return HC == 8 ? MSA_DD(64, 8) : HC == 4 ? MSA_DD(64, 4) : HC == 2 ? MSA_DD(64, 2) : MSA_DD(64, 1);
  return HC == 8 ? MSA_DD(128, 8) : HC == 4 ? MSA_DD(128, 4) : HC == 2 ? MSA_DD(128, 2) : MSA_DD(128, 1);
#undef MSA_DD
}

}  // namespace msa
