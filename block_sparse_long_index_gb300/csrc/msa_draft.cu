// Verification of a tree of drafted tokens against the target's probabilities (msa_verify_tree).
//
// From node 0 on, the children x of the node n are tested in their order with r = max(0, p - c q), where p = probs[n], q =
// draft_probs[n], and c = 0, W = 1 at first: accepted where u q(x) W < r(x); otherwise c grows by W and W becomes the sum
// of r.  That is the rule "reject: replace the target's distribution by max(0, it - q), normalised": with r / W for the
// distribution, max(0, r / W - q) = max(0, p - (c + W) q) / W.  Without q a draft was certain: accepted where u W < r(x),
// otherwise r(x) becomes 0 and W falls by it.  The next token is drawn from the r of the node where the walk ends.
//
// Bound: HBM, one row of p and of q a sequence (a node whose drafts are accepted is left after reading one element of
// each), and more passes over it, from L2, for each further rejection at the node; a few sequences by latency.  A cluster of
// 8 CTAs a sequence: each of its warps has one run of the vocabulary, a pass over a row leaves every run's sum in shared
// memory, and the last pass's sums find the run, then the token, without another pass over the row.
//
// Which token is drawn hangs on comparisons of sums, and a vocabulary may be long: each difference p - c q is worked out as
// an fp32 and its error and counted in units of 2^-58 (exactly from p = 2^-35 on), and the counts are added as integers.
// They add up the same in any order and however a row is split, so that a tree's outcome does not hang on the batch it is
// in, and the sum of V tokens is off by V 2^-59 at most.  (64-bit floating point would be bound by the few units for it;
// fp32 sums draw another token in one of a thousand cases at 128000 tokens.)
//
// Measured: 64 trees of 24 nodes over 128000 tokens 53 us (0.19 of HBM; 47 us with the rows in L2, 17 us where one pass is all:
// a few passes in a row, and the decision between two of them); one tree of 6 over 50001 tokens 12 to 13 us.
#include <math.h>

#include "msa_common.cuh"
#include "msa_sm100.cuh"

namespace msa {

namespace {

constexpr int kCluster = 8;
constexpr int kMaxNodes = 64;
constexpr int kFly = 2;  // vectors of each row that a lane has in flight (64 trees, rows in L2: 1 to 4 take 55, 47, 51, 53 us)
constexpr double kUnit = 288230376151711744.0;           // 2^58
constexpr long long kMost = (1ll << 62) - 1;             // where sums stay: 16, far above a distribution's

// A probability: what is not a positive finite number counts as 0.
__device__ __forceinline__ float prob(float x) { return x > 0.f && x <= 3.402823466e38f ? x : 0.f; }

// Sums of counts of what is no distribution stop at kMost, in any order (all counts are 0 or more).
__device__ __forceinline__ long long add_up(long long a, long long b) { return min(a + b, kMost); }
__device__ __forceinline__ long long warp_sum(long long d) {  // (by pieces of 22 bits, whose sums fit 32)
  constexpr uint32_t kPiece = (1u << 22) - 1u, kTop = 1u << 18;
  const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)d & kPiece), b = __reduce_add_sync(0xffffffffu, (uint32_t)(d >> 22) & kPiece);
  const uint32_t c = __reduce_add_sync(0xffffffffu, (uint32_t)(d >> 44));
  return min(((long long)min(c, kTop) << 44) + ((long long)b << 22) + a, kMost);
}
// The sum of the warp's lanes up to this one.
__device__ __forceinline__ long long warp_scan(long long d) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, d, o);
    if (lane >= o) d = add_up(d, t);
  }
  return d;
}

// x + err, 0 <= x <= 2 and |err| <= 2^-22, in units of 2^-58.  Adding 1.5 2^(23 - k) rounds to a multiple of 2^-k that is
// found in the sum's last bits; what is left goes on to the next k: 21, 44, 58.  err joins in at the second step, and what is
// left of both is added in fp32 (to 2^-68).  Only the last step rounds.
constexpr float kStep1 = 6.f, kStep2 = 7.152557373046875e-7f, kStep3 = 4.3655745685100555e-11f;  // 1.5 2^2, 2^-21, 2^-35
constexpr uint32_t kBits1 = 0x40C00000u, kBits2 = 0x35400000u, kBits3 = 0x2E400000u;             // their bits
constexpr int kShift1 = 58 - 21, kShift2 = 58 - 44;
__device__ __forceinline__ long long counted(float x, float err) {
  const float t = __fadd_rn(x, kStep1), r = __fsub_rn(x, __fsub_rn(t, kStep1));
  const float u = __fadd_rn(r, kStep2), s = __fsub_rn(r, __fsub_rn(u, kStep2));
  const float eu = __fadd_rn(err, kStep2), es = __fsub_rn(err, __fsub_rn(eu, kStep2));
  const float w = __fadd_rn(__fadd_rn(s, es), kStep3);
  return (int)(__float_as_uint(t) - kBits1) * (1ll << kShift1) +
         (int)(__float_as_uint(u) + __float_as_uint(eu) - 2 * kBits2) * (1ll << kShift2) + (int)(__float_as_uint(w) - kBits3);
}

struct VerifyArgs {
  const float *probs, *draft_probs;
  const int32_t *tokens, *parents, *tree_len;
  const float *u, *u_last;
  int32_t *path, *n_path, *next;
  int B, T;
  int64_t V;
  bool report;  // one CTA looks over the whole call's trees and writes the status
};

__device__ __forceinline__ int nodes_of(const VerifyArgs& a, int b, bool& bad) {
  const int t = a.tree_len ? a.tree_len[b] : a.T;
  if (t < 0 || t > a.T) {
    bad = true;
    return 0;
  }
  return t;
}
// Whether node j > 0 of sequence b can be reached, as its parent and token are; otherwise it is passed over.
__device__ __forceinline__ bool offered(const VerifyArgs& a, int b, int j, int& parent, int& token, bool& bad) {
  parent = a.parents[(int64_t)b * a.T + j];
  token = a.tokens[(int64_t)b * a.T + j];
  if (parent < -1 || parent >= j || (parent >= 0 && (token < 0 || (int64_t)token >= a.V))) {
    bad = true;
    return false;
  }
  return parent >= 0;
}

__device__ __forceinline__ long long remote_sum(const long long* p, uint32_t rank) {
  long long x;
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(x) : "r"(at) : "memory");
  return x;
}

// How the difference of a row's elements is taken.
enum Form {
  kPlain,  // p
  kOnce,   // p - q: the first rejection, c = 1
  kTimes,  // p - c q, c = ch + cl
};
// p - c q of clean p and q as an fp32 and its error (exact but for the last bits of cl q); false where it is not positive.
// Where it is, p is at least c q, so that the error of p - t is (p - s) - t.
template <Form F>
__device__ __forceinline__ bool rest_of(float p, float q, float ch, float cl, float& x, float& err) {
  if (F == kPlain) {
    x = p;
    err = 0.f;
    return p > 0.f;
  }
  if (F == kOnce) {
    x = __fsub_rn(p, q);
    err = __fsub_rn(__fsub_rn(p, x), q);
    return x > 0.f;
  }
  const float t = __fmul_rn(ch, q), te = __fmaf_rn(cl, q, __fmaf_rn(ch, q, -t));
  x = __fsub_rn(p, t);
  err = __fsub_rn(__fsub_rn(__fsub_rn(p, x), t), te);
  return __fadd_rn(x, err) > 0.f;
}

// The run [v0, v1) of 4-element vectors that warp `w` of the cluster has; element e of the row is number e + skew of them
// (rows begin anywhere, vectors at multiples of 16 bytes).
struct RowRun {
  int64_t v0, v1;
  int skew;
};
__device__ __forceinline__ RowRun run_of(int64_t row_at, int64_t V, int w, int runs) {
  RowRun r;
  r.skew = (int)(row_at & 3);
  const int64_t vecs = (V + r.skew + 3) / 4, each = (vecs + runs - 1) / runs;
  r.v0 = min(w * each, vecs);
  r.v1 = min(r.v0 + each, vecs);
  return r;
}
// The 4 elements of vector v of a row (base pointer at its element 0), 0 outside it.
__device__ __forceinline__ float4 load_vec(const float* row, int64_t v, int skew, int64_t V) {
  const int64_t e = v * 4 - skew;
  if (e >= 0 && e + 4 <= V) return __ldg(reinterpret_cast<const float4*>(row + e));
  float4 x;
  x.x = e >= 0 && e < V ? row[e] : 0.f;
  x.y = e + 1 >= 0 && e + 1 < V ? row[e + 1] : 0.f;
  x.z = e + 2 >= 0 && e + 2 < V ? row[e + 2] : 0.f;
  x.w = e + 3 >= 0 && e + 3 < V ? row[e + 3] : 0.f;
  return x;
}

// A node's rows and what its rejections left: c (with q), or the tokens that count as 0 (without).
struct Residual {
  const float *p, *q;  // q null: p alone
  float ch, cl;
  const int* out;
  int n_out;
  int64_t V;
  int skew;
  template <Form F>
  __device__ __forceinline__ void load(int64_t v, int64_t v1, float4& a, float4& b) const {
    a = b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (v < v1) {
      a = load_vec(p, v, skew, V);
      if (F != kPlain) b = load_vec(q, v, skew, V);
    }
  }
  template <typename S>
  __device__ __forceinline__ void set(const VerifyArgs& args, const S& step, int64_t at, const int* out_tokens) {
    p = args.probs + at;
    q = step.form == kPlain ? nullptr : args.draft_probs + at;
    ch = step.ch;
    cl = step.cl;
    out = out_tokens;
    n_out = step.n_out;
    V = args.V;
    skew = (int)(at & 3);
  }
  // The vector's r, one by one and clean, in units.  (Where p is a probability nothing is cut off.)
  __device__ __forceinline__ void each(int64_t v, const float4& a, const float4& b, long long (&d)[4]) const {
    constexpr float kErr = 2.384185791015625e-7f;  // 2^-22
    const float pv[4] = {a.x, a.y, a.z, a.w}, qv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x, err;
      const bool on = q ? rest_of<kTimes>(prob(pv[j]), prob(qv[j]), ch, cl, x, err) : rest_of<kPlain>(prob(pv[j]), 0.f, 0.f, 0.f, x, err);
      d[j] = on ? max(counted(fminf(x, 2.f), fminf(fmaxf(err, -kErr), kErr)), 0ll) : 0;
    }
    for (int i = 0; i < n_out; ++i) {
      const int64_t at = (int64_t)out[i] + skew - v * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (at == j) d[j] = 0;
    }
  }
};

// The three steps' last bits of a lane's elements, added up (modulo 2^32; an element of 0 leaves the steps' own bits).
struct Counts {
  uint32_t a, b, c;
};
// A pair of elements, clean: counted() of both at once.
template <Form F>
__device__ __forceinline__ void count2(float p0, float p1, float q0, float q1, float ch, float cl, Counts& n) {
  const uint64_t minus = f2_pack(-1.f, -1.f);
  uint64_t x, err = 0ull;
  if (F == kPlain) {
    x = f2_pack(p0, p1);
  } else if (F == kOnce) {
    const uint64_t p = f2_pack(p0, p1), q = f2_pack(fminf(q0, p0), fminf(q1, p1));  // (p - p: 0, and no error)
    x = f2_fma(q, minus, p);
    err = f2_fma(q, minus, f2_fma(x, minus, p));
  } else {
    float x0, x1, e0, e1;
    if (!rest_of<F>(p0, q0, ch, cl, x0, e0)) x0 = e0 = 0.f;
    if (!rest_of<F>(p1, q1, ch, cl, x1, e1)) x1 = e1 = 0.f;
    x = f2_pack(x0, x1);
    err = f2_pack(e0, e1);
  }
  auto add_bits = [](uint32_t& sum, uint64_t v) { sum += (uint32_t)v + (uint32_t)(v >> 32); };
  const uint64_t t = f2_add(x, f2_pack(kStep1, kStep1)), r = f2_fma(f2_add(t, f2_pack(-kStep1, -kStep1)), minus, x);
  const uint64_t u = f2_add(r, f2_pack(kStep2, kStep2));
  uint64_t s = f2_fma(f2_add(u, f2_pack(-kStep2, -kStep2)), minus, r);
  add_bits(n.a, t);
  add_bits(n.b, u);
  if (F != kPlain) {
    const uint64_t eu = f2_add(err, f2_pack(kStep2, kStep2));
    s = f2_add(s, f2_fma(f2_add(eu, f2_pack(-kStep2, -kStep2)), minus, err));
    add_bits(n.b, eu);
  }
  add_bits(n.c, f2_add(s, f2_pack(kStep3, kStep3)));
}

// A lane's sum over the vectors v0 + lane, + 32, .. below v1.  A value above 1 sends the lane through its vectors again, one
// by one.
template <Form F>
__device__ __forceinline__ long long lane_sum(const Residual& r, int64_t v0, int64_t v1) {
  constexpr uint32_t kEach = 4 * kFly, kTimesB = F == kPlain ? 1 : 2;
  constexpr int kFlush = 256 / kEach;  // rounds whose counts fit 32 bits: 256 elements of 2^21 and of 2^22 + 2^21
  const int lane = threadIdx.x & 31;
  float most = 0.f;
  long long sum = 0;
  for (int64_t v = v0 + lane; v < v1;) {
    Counts n = {0u, 0u, 0u};
    uint32_t rounds = 0;
    for (; rounds < kFlush && v < v1; ++rounds, v += 32 * kFly) {
      float4 a[kFly], b[kFly];
#pragma unroll
      for (int u = 0; u < kFly; ++u) r.load<F>(v + 32 * u, v1, a[u], b[u]);
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        float p[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, q[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
        if (F == kPlain)
          for (int i = 0; i < r.n_out; ++i) {
            const int64_t at = (int64_t)r.out[i] + r.skew - (v + 32 * u) * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (at == j) p[j] = 0.f;
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p[j] = fmaxf(p[j], 0.f), q[j] = fmaxf(q[j], 0.f);  // (a NaN as 0)
          most = fmaxf(most, F == kPlain ? p[j] : fmaxf(p[j], q[j]));
        }
        count2<F>(p[0], p[1], q[0], q[1], r.ch, r.cl, n);
        count2<F>(p[2], p[3], q[2], q[3], r.ch, r.cl, n);
      }
    }
    n.a -= rounds * (kEach * kBits1);
    n.b -= rounds * (kEach * kTimesB * kBits2);
    n.c -= rounds * (kEach * kBits3);
    sum = add_up(sum, min((int)n.a, 1 << 24) * (1ll << kShift1) + (int)n.b * (1ll << kShift2) + (int)n.c);
  }
  if (!(most <= 1.f)) {  // no distribution, or an infinity
    sum = 0;
    for (int64_t v = v0 + lane; v < v1; v += 32) {
      float4 a, b;
      r.load<F>(v, v1, a, b);
      long long d[4];
      r.each(v, a, b, d);
      sum = add_up(sum, add_up(add_up(d[0], d[1]), add_up(d[2], d[3])));
    }
  }
  return sum;
}

// What a CTA does next: one thread's decision, in 64 bits (all threads of a CTA would queue for the few units there are
// for that: with them the smallest call took 25 us).
struct Step {
  int node, n_out, pass;  // pass: sum the residual of `node`; otherwise the walk is over
  int form;
  float ch, cl;
};

// THREADS: 1024 where that leaves a CTA an SM, fewer where several CTAs have to share one.
template <int THREADS>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(THREADS, 1024 / THREADS) verify_kernel(VerifyArgs a, DeviceStatus* st) {
  constexpr int kWarps = THREADS / 32, kRuns = kCluster * kWarps;
  __shared__ int token_s[kMaxNodes], path_s[kMaxNodes], out_s[kMaxNodes];
  __shared__ float p_s[kMaxNodes], q_s[kMaxNodes], u_s[kMaxNodes];
  __shared__ unsigned long long kids_s[kMaxNodes];
  __shared__ long long seg_s[2][kWarps], cta_s[2];  // sums of the warps' runs, and of the CTA's, by pass
  __shared__ long long all_s[kCluster];              // of all the cluster's CTAs, of the last pass
  __shared__ Step step_s;
  __shared__ int n_path_s;
  __shared__ long long target_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / kCluster, rank = (int)cluster_rank();
  bool bad = false;
  const int T = nodes_of(a, b, bad);
  if (tid < kMaxNodes) kids_s[tid] = 0ull;
  __syncthreads();
  if (tid < T) {
    int parent = -1, token = 0;
    float p = 0.f, q = 1.f;
    if (tid > 0 && offered(a, b, tid, parent, token, bad)) {
      const int64_t at = ((int64_t)b * a.T + parent) * a.V + token;
      p = prob(a.probs[at]);
      if (a.draft_probs) q = prob(a.draft_probs[at]);
      atomicOr(&kids_s[parent], 1ull << tid);
    }
    token_s[tid] = token;
    p_s[tid] = p;
    q_s[tid] = q;
    u_s[tid] = a.u[(int64_t)b * a.T + tid];
  }
  if (bad && !a.report && rank == 0) raise_error(st, kErrBadIndex, 14u);
  __syncthreads();

  // ---- the walk: thread 0's state, from pass to pass (the CTAs of the cluster decide alike)
  int n_path = 0, node = 0, n_out = 0, passes = 0;
  unsigned long long kids = kids_s[0];
  double c = 0.0, W = 1.0;
  bool summed = false;  // whether the last pass's sums are those of the present residual
  long long total = 0;  // of the last pass; every thread's
  const float u_last = tid == 0 ? a.u_last[b] : 0.f;
  if (tid == 0 && T > 0) path_s[n_path++] = 0;
  while (T > 0) {
    if (tid == 0) {
      Step step;
      step.pass = 0;
      if (passes && summed) W = (double)total / kUnit;  // (a pass after a rejection; not read after another one)
      while (kids) {
        const int j = __ffsll((long long)kids) - 1;
        kids &= kids - 1;
        double rx;
        bool yes;
        if (a.draft_probs) {
          rx = fmax((double)p_s[j] - c * (double)q_s[j], 0.0);
          yes = (double)q_s[j] * (double)u_s[j] * W < rx;
        } else {
          rx = (double)p_s[j];
          for (int i = 0; i < n_out; ++i)
            if (out_s[i] == token_s[j]) rx = 0.0;
          yes = (double)u_s[j] * W < rx;
        }
        if (yes) {
          node = j;
          kids = kids_s[j];
          c = 0.0;
          W = 1.0;
          n_out = 0;
          summed = false;
          path_s[n_path++] = j;
        } else if (a.draft_probs) {
          c += W;
          step.pass = 1;
          break;
        } else {
          out_s[n_out++] = token_s[j];
          W -= rx;
          summed = false;
        }
      }
      if (!step.pass && !summed) step.pass = 1;  // the walk is over: what the next token is drawn from
      else if (!step.pass && total <= 0 && (c > 0.0 || n_out)) {  // nothing is left (p = q to the last bit): the target's own
        c = 0.0;
        n_out = 0;
        step.pass = 1;
      }
      if (step.pass) summed = true;
      step.node = node;
      step.n_out = n_out;
      step.form = !a.draft_probs || !(c > 0.0) ? kPlain : c == 1.0 ? kOnce : kTimes;
      step.ch = (float)c;
      step.cl = (float)(c - (double)step.ch);
      step_s = step;
      n_path_s = n_path;
    }
    __syncthreads();
    if (!step_s.pass) break;
    // ---- a pass: the residual's sum over the cluster
    {
      Residual r;
      const int64_t at = ((int64_t)b * a.T + step_s.node) * a.V;
      r.set(a, step_s, at, out_s);
      const RowRun run = run_of(at, a.V, rank * kWarps + warp, kRuns);
      long long d = step_s.form == kPlain ? lane_sum<kPlain>(r, run.v0, run.v1)
                    : step_s.form == kOnce ? lane_sum<kOnce>(r, run.v0, run.v1)
                                           : lane_sum<kTimes>(r, run.v0, run.v1);
      d = warp_sum(d);
      if (lane == 0) seg_s[passes & 1][warp] = d;
      __syncthreads();
      if (warp == 0) {
        d = warp_sum(lane < kWarps ? seg_s[passes & 1][lane] : 0);
        if (lane == 0) cta_s[passes & 1] = d;
      }
      cluster_sync();  // (and whoever read the buffer two passes ago is done)
      if (tid < kCluster) all_s[tid] = remote_sum(&cta_s[passes & 1], tid);
      __syncthreads();
      total = 0;
#pragma unroll
      for (int k = 0; k < kCluster; ++k) total = add_up(total, all_s[k]);
      ++passes;
    }
  }
  if (rank == 0) {
    const int n = T > 0 ? n_path_s : 0;
    for (int i = tid; i < a.T; i += THREADS) a.path[(int64_t)b * a.T + i] = i < n ? path_s[i] : -1;
    if (tid == 0) a.n_path[b] = n;
  }
  // ---- the token: the CTA, the warp's run, the vector and the element at which the running sum first exceeds the target
  if (T == 0 || total <= 0) {
    if (rank == 0 && tid == 0) a.next[b] = -1;
  } else {
    if (tid == 0) {
      float ul = u_last;
      ul = ul > 0.f ? fminf(ul, 0.99999994f) : 0.f;  // (a NaN counts as 0)
      target_s = (long long)((double)ul * (double)total);  // a whole sum exceeds u total where it exceeds its whole part
    }
    __syncthreads();
    const long long target = target_s;
    const int buf = (passes - 1) & 1;
    long long before = 0;
    int k = 0;
    bool done = false;
#pragma unroll
    for (int i = 0; i < kCluster; ++i) {
      const long long x = all_s[i];
      if (!done && add_up(before, x) > target) k = i, done = true;
      if (!done) before = add_up(before, x);
    }
    if (done && k == rank) {  // (it is: the sums add up to the total)
      // the warps' runs likewise, a lane each
      // the first lane whose sum, with those of the lanes before it and `at`, exceeds the target (-1: none); `at` grows to
      // what comes before that lane, or by all lanes
      auto first_past = [&](long long of_lane, long long& at) {
        const long long upto = add_up(at, warp_scan(of_lane));
        const int n = __ffs(__ballot_sync(0xffffffffu, upto > target)) - 1;
        const long long below = __shfl_sync(0xffffffffu, upto, n < 0 ? 31 : n > 0 ? n - 1 : 0);
        if (n) at = below;
        return n;
      };
      const int w = first_past(lane < kWarps ? seg_s[buf][lane] : 0, before);
      // all warps take a part of that run each: the part, then its element.  (One warp through the whole run: 7 us more for 64
      // trees.)
      const Step step = step_s;
      Residual r;
      const int64_t at = ((int64_t)b * a.T + step.node) * a.V;
      r.set(a, step, at, out_s);
      const RowRun run = run_of(at, a.V, rank * kWarps + w, kRuns);
      const int64_t each = ((run.v1 - run.v0 + kWarps - 1) / kWarps + 31) / 32 * 32;
      const int64_t first_v = min(run.v0 + warp * each, run.v1), end_v = min(first_v + each, run.v1);
      auto load = [&](int64_t v, long long (&d)[4]) {
        float4 pa, qa;
        if (r.q) r.load<kTimes>(v, end_v, pa, qa);
        else r.load<kPlain>(v, end_v, pa, qa);
        r.each(v, pa, qa, d);
        return add_up(add_up(d[0], d[1]), add_up(d[2], d[3]));
      };
      long long d[4], sum = 0;
#pragma unroll 4
      for (int64_t v = first_v + lane; v < end_v; v += 32) sum = add_up(sum, load(v, d));
      sum = warp_sum(sum);
      if (lane == 0) seg_s[buf ^ 1][warp] = sum;  // (the pass before the last one's are read)
      __syncthreads();
      const long long part = lane < kWarps ? seg_s[buf ^ 1][lane] : 0;
      sum = before;
      if (first_past(part, sum) == warp) {  // (there is one: the parts add up to the run)
        int64_t hit = -1;
        for (int64_t v0 = first_v; v0 < end_v && hit < 0; v0 += 32) {
          const int64_t v = v0 + lane;
          const long long of_lane = load(v, d);
          const int at_lane = first_past(of_lane, sum);
          if (at_lane >= 0) {
            long long x = sum;  // (of lane at_lane; the others' results are not looked at)
            int64_t e = -1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x = add_up(x, d[j]);
              if (e < 0 && x > target) e = v * 4 - r.skew + j;
            }
            hit = __shfl_sync(0xffffffffu, e, at_lane);
          }
        }
        if (lane == 0) a.next[b] = (int32_t)hit;
      }
    }
  }
  if (a.report && blockIdx.x == kCluster - 1) {
    bad = false;
    for (int i = tid; i < a.B * a.T; i += THREADS) {
      const int s = i / a.T, j = i - s * a.T;
      int x, y;
      if (j < nodes_of(a, s, bad) && j > 0) offered(a, s, j, x, y, bad);
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
      st->flags = bad ? kErrBadIndex : 0u;
      st->first_code = bad ? 14u : 0u;
    }
  }
  cluster_sync();  // no CTA leaves while another reads its sums
}

}  // namespace

// The status is written by one CTA of the kernel while the trees are few; otherwise it is cleared before.
bool verify_reports(int B, int T) { return (int64_t)B * T <= 8192; }

cudaError_t launch_verify(const float* probs, const float* draft_probs, const int32_t* tokens, const int32_t* parents,
                          const int32_t* tree_len, const float* u, const float* u_last, int B, int T, int64_t V, int32_t* path,
                          int32_t* n_path, int32_t* next, DeviceStatus* st, cudaStream_t s) {
  VerifyArgs a;
  a.probs = probs;
  a.draft_probs = draft_probs;
  a.tokens = tokens;
  a.parents = parents;
  a.tree_len = tree_len;
  a.u = u;
  a.u_last = u_last;
  a.path = path;
  a.n_path = n_path;
  a.next = next;
  a.B = B;
  a.T = T;
  a.V = V;
  a.report = verify_reports(B, T);
  // CTAs of all sequences together on the GPU, where that is possible
  const int64_t ctas = (int64_t)B * kCluster, sms = num_sms();
  if (ctas <= sms) verify_kernel<1024><<<(unsigned)ctas, 1024, 0, s>>>(a, st);
  else if (ctas <= 2 * sms) verify_kernel<512><<<(unsigned)ctas, 512, 0, s>>>(a, st);
  else verify_kernel<256><<<(unsigned)ctas, 256, 0, s>>>(a, st);
  return cudaGetLastError();
}

}  // namespace msa
