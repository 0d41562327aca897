// What the kernels of a call of tree attention share: its shape, and the partial results that they leave.
#pragma once

#include "msa_internal.h"

namespace msa {

constexpr int kKeysT = 128;  // tokens of a tile

struct TreeShape {
  const int32_t* ctx;       // [B]
  const int32_t* tree_len;  // [B], null: T each
  int64_t cap;
  int B, T, gs, H_kv;
  int RG, RU;          // row groups of a (sequence, K/V head), rows of one
  int groups, rounds;  // see tree_plan
  int ways;            // partials of a (segment, unit)
  int lg;              // log2 of the tokens of an entry of the list that is split into runs (7: tiles)
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
  __device__ __forceinline__ int spans(int b) const {
    int n, t;
    lengths(b, n, t);
    return t ? (int)(((int64_t)n + (1 << lg) - 1) >> lg) : 0;
  }
};

// Scratch of a call: what the context kernel leaves for the joining one.
struct TreeScratch {
  int64_t* starts;       // [B + 1] entries of the list before each sequence, then those of a run
  unsigned int* errors;  // [CTAs] flags each met
  // [slots][D / 8][RU][8] (a lane of the context kernel has a row, one of the joining kernel channels); slot =
  // ((sequence + group) ways + way) units + unit, which no two segments share
  float* part_o;
  float2* part_ml;       // [slots][RU] maximum (log2 units) and sum
};
// Channel ch of row r in a slot's partial O.
__device__ __forceinline__ int part_at(int RU, int r, int ch) { return ((ch >> 3) * RU + r) * 8 + (ch & 7); }

// The context over 4-bit pages for few rows a K/V head (msa_tree_few.cu): most rows, most K/V heads; CTAs and partials.
constexpr int kFewRows = 32, kFewHeads = 8;
int few_ctas(int rows);
int few_ways(int H_kv);
int few_lg(int B, int64_t cap);
cudaError_t launch_tree_few(const void* q, const TreeShape& sh, const CacheMap& map, const Kv4Pool& pool, int d, float scale_log2,
                            const TreeScratch& w, DeviceStatus* st, cudaStream_t s);

}  // namespace msa
