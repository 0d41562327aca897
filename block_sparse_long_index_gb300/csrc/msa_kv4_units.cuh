// Walking a 4-bit paged cache in units of 16 tokens: the ring's stages that TMA fills (codes of a step's units, then their
// scales), and how a lane's codes in them become mma.sync fragments without passing through shared memory again.
#pragma once

#include "msa_kv4.cuh"

namespace msa {
namespace kv4 {

constexpr int kUnit = 16;
constexpr int kDecWarps = 8;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr float kLazy = 8.0f;  // log2 units a row maximum may grow before O is rescaled
constexpr int kMaxStages = 8;
constexpr uint32_t kNaNRaw = (kScaleNaN << 4) + kSubScaleBias;  // M of the NaN scale before it is made NaN

template <int D>
struct Tile {
  static constexpr int CB = D / 2;           // bytes of a head row's codes, and the span of the TMA swizzle
  static constexpr int BYTES = kUnit * CB;   // a unit's codes of one head
  // token of row i of S^T (rows 8 .. 15: 8 more).  d = 128 (64-byte rows, 16-byte piece p at p ^ (token / 2 % 4)):
  // even rows 0 1 4 5, odd rows 3 2 7 6; d = 64 (32-byte rows, piece p at p ^ (token / 4 % 2)): 0 1 2 3 and 6 7 4 5.
  __device__ static __forceinline__ int perm(int i) {
    const int c = (i >> 1) & 3;
    const int even = D == 128 ? c + 2 * (c >> 1) : c;
    return (i & 8) + ((i & 1) == 0 ? even : D == 128 ? (even ^ 3) : 4 + ((c + 2) & 3));
  }
  // where byte b of token t's codes sits in the tile
  __device__ static __forceinline__ int at(int t, int b) {
    return t * CB + (b ^ (16 * (D == 128 ? (t >> 1) & 3 : (t >> 2) & 1)));
  }
};

// Bytes of a stage: K and V codes of the step's 16 (unit, head) tiles, then its 2 TW units' scales of every head.
__host__ __device__ constexpr int stage_bytes(int d, int tw, int H_kv) {
  return (32 * kUnit * (d / 2) + 4 * tw * kUnit * H_kv * kGroups + 1023) / 1024 * 1024;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, int32_t w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Reads of the ring by shared-memory address (a generic pointer would cost 64-bit arithmetic for each).
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.u8 %0, [%1];\n" : "=r"(x) : "r"(a));
  return x;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "a load's width");
  if constexpr (N == 1) asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(w[0]) : "r"(a));
  if constexpr (N == 2) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
}
__device__ __forceinline__ uint32_t hmax2_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Units of a CTA's run: a multiple of a step's, so that none of its warps starts idle.
__device__ __forceinline__ int64_t quota_of(int64_t total, int n_cta, int step) {
  return ((total + n_cta - 1) / n_cta + step - 1) / step * step;
}

}  // namespace kv4
}  // namespace msa
