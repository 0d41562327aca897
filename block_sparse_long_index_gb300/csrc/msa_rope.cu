// Rotary positions: rows turned by themselves (msa_rope), and rows of new tokens on their way into a paged cache
// (msa_append_paged, msa_append_paged_kv4).
//
// A pair (a, b) of channels at position p with frequency f turns by the angle p f:
//   a' = a cos - b sin,  b' = b cos + a sin.
// The frequency is given as F = f / 2 pi in 2^-64 turns, so that p F modulo 2^64 is the angle modulo a turn, exactly,
// whatever p is: two integer multiplications instead of a reduction in 64-bit floating point (at p = 2^20 an fp32
// angle would be off by 0.03).  cos and sin are worked out once a (token, pair) and shared by all heads.
//
// Bound: HBM, rows in and out once.  Measured: 32768 rows of 64 heads, d = 128, fp32, half of the channels turned: 328 us,
// 6.55 TB/s (0.98 of the measured copy rate), bf16 and all of them 200 us, 5.4 TB/s (0.80); 48 rows of 32 heads: 5 us, a
// launch's latency and one round trip.
#include <math.h>

#include "msa_kv4.cuh"
#include "msa_rows.cuh"

namespace msa {

namespace {

using namespace kv4;

constexpr int kWarps = kRowThreads / 32;
constexpr int kFly = 4;       // 16-byte reads a thread has in flight
constexpr int kMaxToks = 16;  // tokens of a CTA

// cos and sin of 2^-64 ph turns, each within 2^-24 of the exact value (half a step from 1/2 on, and what the last sum adds).  The
// angle is reduced to +-1/8 turn around the
// nearest quarter; there the Taylor polynomials, whose first missing terms are below 2^-37, are summed from the small
// end with the roundings of the leading terms carried along (their products written as an fp32 and its error).
__device__ __forceinline__ void cos_sin(uint64_t ph, float& c, float& s) {
  const uint32_t quarter = (uint32_t)((ph + (1ull << 61)) >> 62);
  const int64_t r = (int64_t)(ph - ((uint64_t)quarter << 62));  // +-2^61
  const int32_t h = (int32_t)(r >> 32);
  const float f1 = __int2float_rn(h);
  const float f2 = __fmaf_rn(__uint2float_rn((uint32_t)r), 2.3283064365386963e-10f, __int2float_rn(h - (int32_t)f1));
  // 2 pi 2^-32 as a sum of two fp32
  constexpr double kUnit = 6.283185307179586476925286766559 / 4294967296.0;
  constexpr float kHi = (float)kUnit, kLo = (float)(kUnit - (double)(float)kUnit);
  const float a = __fmul_rn(f1, kHi);
  const float al = __fmaf_rn(f2, kHi, __fmaf_rn(f1, kLo, __fmaf_rn(f1, kHi, -a)));  // the angle is a + al
  const float u = __fmul_rn(a, a), ul = __fmaf_rn(2.f * a, al, __fmaf_rn(a, a, -u));
  float p = __fmaf_rn(u, -2.50521083854417e-8f, 2.75573192239859e-6f);  // -1/11!, 1/9!
  p = __fmaf_rn(u, p, -1.98412698412698e-4f);
  p = __fmaf_rn(u, p, 8.33333333333333e-3f);
  p = __fmaf_rn(u, p, -1.66666666666667e-1f);
  const float sn = __fadd_rn(a, __fmaf_rn(__fmul_rn(a, u), p, __fmaf_rn(-0.5f * u, al, al)));
  p = __fmaf_rn(u, 2.08767569878681e-9f, -2.75573192239859e-7f);  // 1/12!, -1/10!
  p = __fmaf_rn(u, p, 2.48015873015873e-5f);
  p = __fmaf_rn(u, p, -1.38888888888889e-3f);
  p = __fmaf_rn(u, p, 4.16666666666667e-2f);
  const float w = __fmaf_rn(-0.5f, u, 1.f), we = __fmaf_rn(-0.5f, u, __fsub_rn(1.f, w));
  const float cs = __fadd_rn(w, __fadd_rn(we, __fmaf_rn(__fmul_rn(u, u), p, -0.5f * ul)));
  const bool swap = quarter & 1u;
  c = swap ? sn : cs;
  s = swap ? cs : sn;
  if (quarter == 1u || quarter == 2u) c = -c;
  if (quarter & 2u) s = -s;
}

// The tokens' cos and sin, [n][2][span] (cos, then sin), for the rot / 2 pairs; `sign` -1 turns back.
__device__ __forceinline__ void fill_turns(const Rope& rope, const int32_t* pos, int n, int span, float sign, float* cs) {
  const int half = rope.rot / 2;
  for (int x = threadIdx.x; x < n * half; x += kRowThreads) {
    const int t = x / half, i = x - t * half;
    float c, s;
    cos_sin((uint64_t)(int64_t)pos[t] * rope.turns[i], c, s);
    cs[(2 * t) * span + i] = __fmul_rn(c, rope.factor);
    cs[(2 * t + 1) * span + i] = __fmul_rn(__fmul_rn(s, sign), rope.factor);
  }
}

// a c - b s and b c + a s with three roundings each, as the plain formula has them: turning a row and then storing it
// and storing it turned give equal bits, with or without a fused multiply-add elsewhere.
__device__ __forceinline__ float turn_1(float a, float b, float c, float s) { return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)); }
__device__ __forceinline__ float turn_2(float a, float b, float c, float s) { return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)); }

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// Turns the 8 channels 8 p .. of a row whose `lanes` threads (a power of two, a run of the warp's) hold 8 each.  Every
// lane of the warp takes part.  `c`: the token's cos, its sin `span` further.
__device__ __forceinline__ void turn8(float (&x)[8], int p, int lanes, const Rope& rope, const float* c, int span) {
  if (rope.interleaved) {
    if (16 * p < 2 * rope.rot) {
      const float4 cv = *reinterpret_cast<const float4*>(c + 4 * p), sv = *reinterpret_cast<const float4*>(c + span + 4 * p);
      const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = x[2 * j], b = x[2 * j + 1];
        x[2 * j] = turn_1(a, b, cc[j], ss[j]);
        x[2 * j + 1] = turn_2(a, b, cc[j], ss[j]);
      }
    }
    return;
  }
  const int hp = rope.rot / 16;  // pieces of a half
  const bool first = p < hp, in = p < 2 * hp;
  const int q = !in ? p : first ? p + hp : p - hp, src = ((int)(threadIdx.x & 31u) & ~(lanes - 1)) | q;
  float o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(0xffffffffu, x[j], src);
  if (!in) return;
  float cc[8], ss[8];
  load8(c + 8 * (first ? p : q), cc);
  load8(c + span + 8 * (first ? p : q), ss);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = first ? turn_1(x[j], o[j], cc[j], ss[j]) : turn_2(o[j], x[j], cc[j], ss[j]);
}

__device__ __forceinline__ uint4 ld_once(const void* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }
// Pairs of fp32 with every result rounded as by itself, subnormal ones included.
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t narrow2(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return pack_bf16x2(a, b);
}
__device__ __forceinline__ uint64_t widen2(uint32_t w) { return f2_pack(bf16_lo(w), bf16_hi(w)); }

// turn8 of bf16 rows: the words of a piece, turned and rounded.  (A product with -s is the product with s negated, so
// a c - b s is a c + (-b) s to the last bit.)
__device__ __forceinline__ uint4 turn8_bf16(uint4 w, int p, int lanes, const Rope& rope, const float* c, int span) {
  uint32_t v[4] = {w.x, w.y, w.z, w.w};
  if (rope.interleaved) {
    if (8 * p >= rope.rot) return w;
    const float4 cv = *reinterpret_cast<const float4*>(c + 4 * p), sv = *reinterpret_cast<const float4*>(c + span + 4 * p);
    const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t o = __byte_perm(v[j], v[j] ^ 0x80000000u, 0x1076);  // (-b, a)
      v[j] = narrow2(add2(mul2(widen2(v[j]), f2_pack(cc[j], cc[j])), mul2(widen2(o), f2_pack(ss[j], ss[j]))));
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
  const int hp = rope.rot / 16;  // pieces of a half
  const bool first = p < hp, in = p < 2 * hp;
  const int q = !in ? p : first ? p + hp : p - hp, src = ((int)(threadIdx.x & 31u) & ~(lanes - 1)) | q;
  const uint32_t sign = first ? 0x80008000u : 0u;
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = __shfl_sync(0xffffffffu, v[j], src) ^ sign;
  if (!in) return w;
  const ulonglong2* cp = reinterpret_cast<const ulonglong2*>(c + 8 * (first ? p : q));
  const ulonglong2* sp = reinterpret_cast<const ulonglong2*>(c + span + 8 * (first ? p : q));
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const ulonglong2 cj = cp[j], sj = sp[j];
    v[2 * j] = narrow2(add2(mul2(widen2(v[2 * j]), cj.x), mul2(widen2(o[2 * j]), sj.x)));
    v[2 * j + 1] = narrow2(add2(mul2(widen2(v[2 * j + 1]), cj.y), mul2(widen2(o[2 * j + 1]), sj.y)));
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// The same for a piece of 16 channels, where the halves of the pairs are whole pieces or side by side.
__device__ __forceinline__ void turn16_bf16(uint4 (&w)[2], int p, int lanes, const Rope& rope, const float* c, int span) {
  if (rope.interleaved) {
#pragma unroll
    for (int h = 0; h < 2; ++h) w[h] = turn8_bf16(w[h], 2 * p + h, lanes, rope, c, span);
    return;
  }
  const int hp = rope.rot / 32;  // pieces of a half
  const bool first = p < hp, in = p < 2 * hp;
  const int q = !in ? p : first ? p + hp : p - hp, src = ((int)(threadIdx.x & 31u) & ~(lanes - 1)) | q;
  const uint32_t sign = first ? 0x80008000u : 0u;
  const float* cp = c + 16 * (first ? p : q);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v[4] = {w[h].x, w[h].y, w[h].z, w[h].w}, o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = __shfl_sync(0xffffffffu, v[j], src) ^ sign;
    if (in) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const ulonglong2 cj = reinterpret_cast<const ulonglong2*>(cp + 8 * h)[j], sj = reinterpret_cast<const ulonglong2*>(cp + span + 8 * h)[j];
        v[2 * j] = narrow2(add2(mul2(widen2(v[2 * j]), cj.x), mul2(widen2(o[2 * j]), sj.x)));
        v[2 * j + 1] = narrow2(add2(mul2(widen2(v[2 * j + 1]), cj.y), mul2(widen2(o[2 * j + 1]), sj.y)));
      }
      w[h] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
}
__device__ __forceinline__ uint32_t cvt_e4m3x2(float hi, float lo) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The E4M3 codes of 8 bf16 values times `scale`, as msa_quantize_e4m3 makes them.
__device__ __forceinline__ uint2 e4m3_8(uint4 w, float scale) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  uint32_t p[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = cvt_e4m3x2(__fmul_rn(bf16_hi(v[j]), scale), __fmul_rn(bf16_lo(v[j]), scale));
  return make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
}

// ---------------------------------------------------------------- rows by themselves
// Rows of T (bf16 words or fp32) [N, H, d] turned, or turned back, into y (x itself is allowed).  A warp takes 256
// channels of a token at a time; a row's threads hand one another the other half of their pairs by shuffles.
// Bound: HBM, each row once in and once out.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) rope_kernel(const T* __restrict__ x, int64_t x_stride, T* y, int64_t y_stride,
                                                           int64_t N, int H, int d, const int32_t* __restrict__ positions,
                                                           int toks, float sign, Rope rope) {
  constexpr bool F32 = sizeof(T) == 4;
  __shared__ __align__(16) float cs[kMaxToks * 2 * 128];
  __shared__ int32_t pos[kMaxToks];
  const int64_t i0 = (int64_t)blockIdx.x * toks;
  const int n = (int)min((int64_t)toks, N - i0);
  if ((int)threadIdx.x < n) pos[threadIdx.x] = positions[i0 + threadIdx.x];
  __syncthreads();
  fill_turns(rope, pos, n, 128, sign, cs);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lanes = d / 8;
  const int pieces = H * lanes, chunks = (pieces + 31) / 32, tasks = n * chunks;
  for (int base = warp; base < tasks; base += kWarps * kFly) {
    uint4 w[kFly][F32 ? 2 : 1];
#pragma unroll
    for (int u = 0; u < kFly; ++u) {
      const int task = base + u * kWarps, t = task / chunks, e = (task - t * chunks) * 32 + lane;
#pragma unroll
      for (int j = 0; j < (F32 ? 2 : 1); ++j)
        w[u][j] = task < tasks && e < pieces ? ld_once(x + (i0 + t) * x_stride + e * 8 + 4 * j) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < kFly; ++u) {
      const int task = base + u * kWarps, t = task / chunks, e = (task - t * chunks) * 32 + lane;
      if (task >= tasks) break;  // (uniform in the warp)
      const int p = e & (lanes - 1);
      T* to = y + (i0 + t) * y_stride + e * 8;
      if constexpr (F32) {
        float v[8] = {__uint_as_float(w[u][0].x), __uint_as_float(w[u][0].y), __uint_as_float(w[u][0].z), __uint_as_float(w[u][0].w),
                      __uint_as_float(w[u][1].x), __uint_as_float(w[u][1].y), __uint_as_float(w[u][1].z), __uint_as_float(w[u][1].w)};
        turn8(v, p, lanes, rope, cs + 2 * t * 128, 128);
        if (e >= pieces) continue;
        *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(to + 4) = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        const uint4 v = turn8_bf16(w[u][0], p, lanes, rope, cs + 2 * t * 128, 128);
        if (e < pieces) *reinterpret_cast<uint4*>(to) = v;
      }
    }
  }
}

// ---------------------------------------------------------------- rows into a paged cache
// What a token's rows are made of, in pieces of 8 channels: a warp takes 32 pieces of one kind of a token at a time (a
// chunk), with kFly tokens' in flight.  The kinds have code of their own: with one loop for all of them the choices among
// them were half of the instructions (131072 tokens into 4 bits 324 us, 0.79 of the issue slots).
enum Kind { kQ, kK, kV, kQI, kKI };
constexpr int kSpan = 64;
struct Rows {
  int H_kv;
  uint16_t *k_pool, *v_pool;
  Kv4Pool pool;
};
template <int D, bool KV4, Kind K>
__device__ __forceinline__ void append_kind(const AppendRows& a, const Rows& io, int pieces, int64_t i0, int n,
                                            const int64_t* rows, const float* cs, int& turn) {
  constexpr int LPR = D / 8, LPG = LPR / kGroups;
  constexpr bool idx = K == kQI || K == kKI, pooled = K == kK || K == kV;
  const int lane = threadIdx.x & 31, chunks = (pieces + 31) / 32, tasks = n * chunks;
  const int batches = (tasks + kFly - 1) / kFly;
  const uint16_t* const src = K == kQ ? a.q : K == kK ? a.k : K == kV ? a.v : K == kQI ? a.q_idx : a.k_idx;
  const int64_t stride = K == kQ ? a.q_stride : K == kK ? a.k_stride : K == kV ? a.v_stride : K == kQI ? a.q_idx_stride : a.k_idx_stride;
  for (int batch = turn; batch < batches; batch += kWarps) {
    int c = batch * kFly / n, t = batch * kFly - c * n;  // the tokens of a chunk one after the other
    uint4 w[kFly];
    int tok[kFly], piece[kFly];  // piece -1 - e where this lane has none
#pragma unroll
    for (int u = 0; u < kFly; ++u) {
      const int e = c * 32 + lane;
      const bool on = c < chunks && e < pieces && rows[t] >= 0;
      w[u] = on ? ld_once(src + (i0 + t) * stride + e * 8) : make_uint4(0u, 0u, 0u, 0u);
      tok[u] = t;
      piece[u] = on ? e : -1 - e;
      if (++t == n) t = 0, ++c;
    }
#pragma unroll
    for (int u = 0; u < kFly; ++u) {
      if (batch * kFly + u >= tasks) break;  // (uniform in the warp)
      const bool on = piece[u] >= 0;
      const int e = on ? piece[u] : -1 - piece[u];
      if (K != kV) {
        const int lanes = idx ? a.d_I / 8 : LPR;
        w[u] = turn8_bf16(w[u], e & (lanes - 1), lanes, idx ? a.rope_idx : a.rope, cs + 2 * tok[u] * kSpan, kSpan);
      }
      if (pooled && KV4) {
        const unsigned lanes = ((1u << LPG) - 1u) << (lane & ~(LPG - 1));
        uint32_t code, sb;
        encode8<LPG>(w[u], lanes, code, sb);
        if (on) {
          const int64_t row = rows[tok[u]];
          uint8_t* codes = K == kV ? io.pool.v_codes : io.pool.k_codes;
          uint8_t* scales = K == kV ? io.pool.v_scales : io.pool.k_scales;
          reinterpret_cast<uint32_t*>(codes)[row * (io.H_kv * LPR) + e] = code;
          if (e % LPG == 0) scales[row * (io.H_kv * kGroups) + e / LPG] = (uint8_t)sb;
        }
      } else if (on) {
        const int64_t row = pooled || K == kKI ? rows[tok[u]] : i0 + tok[u];
        const int width = K == kQ ? a.H_q * D : pooled ? io.H_kv * D : K == kQI ? io.H_kv * a.d_I : a.d_I;
        void* to = K == kQ ? a.q_out : K == kK ? io.k_pool : K == kV ? io.v_pool : K == kQI ? a.q_idx_out : a.k_idx_pool;
        const int64_t at = row * width + e * 8;
        if (idx && a.idx_f8) *reinterpret_cast<uint2*>((uint8_t*)to + at) = e4m3_8(w[u], a.idx_scale);
        else *reinterpret_cast<uint4*>((uint16_t*)to + at) = w[u];
      }
    }
  }
  turn = (turn - batches % kWarps + kWarps) % kWarps;  // the next kind begins where this one ended
}

// K or V into a 4-bit pool with 16 channels a thread: what a group's threads each work out for themselves (its scale), and
// a piece's place, is done half as often as with 8.  The halves of K's pairs have to be whole pieces: rot a multiple of 32,
// or pairs side by side.
__host__ __device__ constexpr bool wide_turn(int rot, bool interleaved) { return interleaved || rot % 32 == 0; }
template <int D, Kind K>
__device__ __forceinline__ void append_codes(const AppendRows& a, const Rows& io, int64_t i0, int n, const int64_t* rows,
                                             const float* cs, int& turn) {
  constexpr int LPR = D / 16, LPG = LPR / kGroups, FLY = kFly / 2;
  const int lane = threadIdx.x & 31, pieces = io.H_kv * LPR, chunks = (pieces + 31) / 32, tasks = n * chunks;
  const int batches = (tasks + FLY - 1) / FLY;
  const uint16_t* const src = K == kK ? a.k : a.v;
  const int64_t stride = K == kK ? a.k_stride : a.v_stride;
  uint8_t* const codes = K == kV ? io.pool.v_codes : io.pool.k_codes;
  uint8_t* const scales = K == kV ? io.pool.v_scales : io.pool.k_scales;
  const unsigned group = ((1u << LPG) - 1u) << (lane & ~(LPG - 1));
  for (int batch = turn; batch < batches; batch += kWarps) {
    int c = batch * FLY / n, t = batch * FLY - c * n;  // the tokens of a chunk one after the other
    uint4 w[FLY][2];
    int tok[FLY], piece[FLY];  // piece -1 - e where this lane has none
#pragma unroll
    for (int u = 0; u < FLY; ++u) {
      const int e = c * 32 + lane;
      const bool on = c < chunks && e < pieces && rows[t] >= 0;
      const uint16_t* p = src + (i0 + t) * stride + e * 16;
      w[u][0] = on ? ld_once(p) : make_uint4(0u, 0u, 0u, 0u);
      w[u][1] = on ? ld_once(p + 8) : make_uint4(0u, 0u, 0u, 0u);
      tok[u] = t;
      piece[u] = on ? e : -1 - e;
      if (++t == n) t = 0, ++c;
    }
#pragma unroll
    for (int u = 0; u < FLY; ++u) {
      if (batch * FLY + u >= tasks) break;  // (uniform in the warp)
      const bool on = piece[u] >= 0;
      const int e = on ? piece[u] : -1 - piece[u];
      if (K == kK) turn16_bf16(w[u], e & (LPR - 1), LPR, a.rope, cs + 2 * tok[u] * kSpan, kSpan);
      uint2 code;
      uint32_t sb;
      encode16<LPG>(w[u], group, code, sb);
      if (on) {
        const int64_t row = rows[tok[u]];
        reinterpret_cast<uint2*>(codes)[row * pieces + e] = code;
        if (e % LPG == 0) scales[row * (io.H_kv * kGroups) + e / LPG] = (uint8_t)sb;
      }
    }
  }
  turn = (turn - batches % kWarps + kWarps) % kWarps;
}

// A CTA takes `toks` packed tokens: it looks up their places, works out their cos and sin, and its warps then go
// through the tokens' chunks with four reads in flight.  K is rounded to bf16 once turned, then stored or quantized, so
// that the cache holds what turning and storing in two calls would leave.  Bound: HBM, rows in and out once; few
// tokens by the launch and the chain look-up, angles, rows.  Measured, 131072 tokens of 8 heads, d = 128, with index keys:
// into bf16 pages 179 us (0.89 of the copy rate), into 4-bit pages 207 us (0.49), where the issue slots are busy with the
// angles, the turns and the codes (250 us with 8 channels a thread for K and V too); 48 tokens with 32 query heads: 7 us.
template <int D, bool KV4>
__global__ void __launch_bounds__(kRowThreads) append_kernel(AppendRows a, int64_t N, int toks, RowMap map, uint16_t* k_pool,
                                                             uint16_t* v_pool, Kv4Pool pool, DeviceStatus* st) {
  constexpr int LPR = D / 8;
  __shared__ __align__(16) float cs[2][kMaxToks * 2 * kSpan];  // of the attention's rows, of the index rows
  __shared__ int64_t rows[kRowThreads];
  __shared__ int32_t pos[kRowThreads];
  const int64_t i0 = (int64_t)blockIdx.x * toks;
  look_up(map, N, i0, toks, -1, rows, st, pos);
  const int n = (int)min((int64_t)toks, N - i0);
  if (a.positions && (int)threadIdx.x < n) pos[threadIdx.x] = a.positions[i0 + threadIdx.x];
  __syncthreads();
  fill_turns(a.rope, pos, n, kSpan, 1.f, cs[0]);
  if (a.rope_idx_own) fill_turns(a.rope_idx, pos, n, kSpan, 1.f, cs[1]);
  __syncthreads();
  const Rows io = {a.H_kv, k_pool, v_pool, pool};
  int turn = threadIdx.x >> 5;  // a batch of one kind after the other goes to the warps in turn
  if (a.q) append_kind<D, KV4, kQ>(a, io, a.H_q * LPR, i0, n, rows, cs[0], turn);
  if (KV4 && wide_turn(a.rope.rot, a.rope.interleaved)) append_codes<D, kK>(a, io, i0, n, rows, cs[0], turn);
  else append_kind<D, KV4, kK>(a, io, a.H_kv * LPR, i0, n, rows, cs[0], turn);
  if (KV4) append_codes<D, kV>(a, io, i0, n, rows, cs[0], turn);
  else append_kind<D, KV4, kV>(a, io, a.H_kv * LPR, i0, n, rows, cs[0], turn);
  const float* cs_idx = cs[a.rope_idx_own ? 1 : 0];
  if (a.q_idx) append_kind<D, KV4, kQI>(a, io, a.H_kv * (a.d_I / 8), i0, n, rows, cs_idx, turn);
  if (a.k_idx) append_kind<D, KV4, kKI>(a, io, a.d_I / 8, i0, n, rows, cs_idx, turn);
}

// Tokens of a CTA: more than one only where the CTAs still fill the GPU four times.
int toks_of(int64_t N) {
  const int64_t t = N / ((int64_t)4 * num_sms());
  return t > kMaxToks ? kMaxToks : t < 1 ? 1 : (int)t;
}

}  // namespace

cudaError_t launch_rope(const void* x, int64_t x_stride, void* y, int64_t y_stride, int64_t N, int H, int d, bool f32,
                        const int32_t* positions, const Rope& rope, bool inverse, cudaStream_t s) {
  const int toks = toks_of(N);
  const unsigned grid = (unsigned)ceil_div(N, toks);
  const float sign = inverse ? -1.f : 1.f;
  if (f32)
    rope_kernel<float><<<grid, kRowThreads, 0, s>>>((const float*)x, x_stride, (float*)y, y_stride, N, H, d, positions, toks,
                                                    sign, rope);
  else
    rope_kernel<uint16_t><<<grid, kRowThreads, 0, s>>>((const uint16_t*)x, x_stride, (uint16_t*)y, y_stride, N, H, d, positions,
                                                       toks, sign, rope);
  return cudaGetLastError();
}

cudaError_t launch_append(const AppendRows& rows, int64_t N, const int32_t* cu, int S, const int32_t* pos0,
                          const int32_t* table, int64_t max_pages, void* k_pool, void* v_pool, const Kv4Pool* kv4,
                          int64_t n_pages, int page, int d, DeviceStatus* st, cudaStream_t s) {
  const RowMap map = row_map(cu, S, pos0, table, max_pages, n_pages, page);
  const int toks = toks_of(N);
  auto kern = kv4 ? (d == 64 ? append_kernel<64, true> : append_kernel<128, true>)
                  : (d == 64 ? append_kernel<64, false> : append_kernel<128, false>);
  kern<<<(unsigned)ceil_div(N, toks), kRowThreads, 0, s>>>(rows, N, toks, map, (uint16_t*)k_pool, (uint16_t*)v_pool,
                                                           kv4 ? *kv4 : Kv4Pool{}, st);
  return cudaGetLastError();
}

}  // namespace msa
