// Verification of a tree of drafted tokens against the target's probabilities (msa_verify_tree).
//
// From node 0 on, the children x of the node n are tested in their order with r = max(0, p - c q), where p = probs[n], q =
// draft_probs[n], and c = 0, W = 1 at first: accepted where u q(x) W < r(x); otherwise c grows by W and W becomes the sum
// of r.  That is the rule "reject: replace the target's distribution by max(0, it - q), normalised": with r / W for the
// distribution, max(0, r / W - q) = max(0, p - (c + W) q) / W.  Without q a draft was certain: accepted where u W < r(x),
// otherwise r(x) becomes 0 and W falls by it.  The next token is drawn from the r of the node where the walk ends.
//
// Bound: HBM, one row of p and of q a sequence (a node whose drafts are accepted is left after reading one element of
// each); a few sequences by latency.  A cluster of 8 CTAs a sequence: each of its 128 warps has one run of the
// vocabulary, a pass over a row leaves every run's sum in shared memory, and the last pass's sums find the run, then the
// token, without another pass over the row.
//
// Which token is drawn hangs on comparisons of sums, so these are held to some 48 bits: each difference p - c q is an fp32
// and its error, summed as such by a lane, and from there in 64 bits.  (64-bit sums throughout would be bound by the few
// 64-bit units; fp32 sums draw another token in one of a thousand cases at 128000 tokens.)
#include <math.h>

#include "msa_common.cuh"

namespace msa {

namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxNodes = 64;

// A probability: what is not a positive finite number counts as 0.
__device__ __forceinline__ float prob(float x) { return x > 0.f && x <= 3.402823466e38f ? x : 0.f; }

// A sum as an fp32 and its error.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x, float err) {
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)), err));
    hi = s;
  }
};

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

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ double remote_double(const double* p, uint32_t rank) {
  double x;
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(x) : "r"(at) : "memory");
  return x;
}

// r of one element: an fp32 and its error, (0, 0) where it is not positive.  c = ch + cl.
__device__ __forceinline__ void rest_of(float p, float q, float ch, float cl, float& x, float& err) {
  p = prob(p);
  q = prob(q);
  const float t = __fmul_rn(ch, q), te = __fmaf_rn(cl, q, __fmaf_rn(ch, q, -t));
  const float s = __fsub_rn(p, t), b = __fsub_rn(s, p);
  const float e = __fsub_rn(__fsub_rn(__fsub_rn(p, __fsub_rn(s, b)), __fadd_rn(t, b)), te);
  const bool on = __fadd_rn(s, e) > 0.f;
  x = on ? s : 0.f;
  err = on ? e : 0.f;
}

// The run [v0, v1) of 4-element vectors that warp `w` of the cluster has; element e of the row is number e + skew of them
// (rows begin anywhere, vectors at multiples of 16 bytes).
struct RowRun {
  int64_t v0, v1;
  int skew;
};
__device__ __forceinline__ RowRun run_of(int64_t row_at, int64_t V, int w) {
  RowRun r;
  r.skew = (int)(row_at & 3);
  const int64_t vecs = (V + r.skew + 3) / 4, each = (vecs + kCluster * kWarps - 1) / (kCluster * kWarps);
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

// The state of a node's residual: c (with q), or the tokens taken out (without).
struct Residual {
  const float *p, *q;  // q null: p alone
  float ch, cl;
  const int* out;  // tokens that count as 0
  int n_out;
  int64_t V;
  int skew;
  __device__ __forceinline__ void at(int64_t v, float (&x)[4], float (&err)[4]) const {
    const float4 a = load_vec(p, v, skew, V);
    const float pv[4] = {a.x, a.y, a.z, a.w};
    if (q) {
      const float4 b = load_vec(q, v, skew, V);
      const float qv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) rest_of(pv[j], qv[j], ch, cl, x[j], err[j]);
      return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = prob(pv[j]), err[j] = 0.f;
    for (int i = 0; i < n_out; ++i) {
      const int64_t d = (int64_t)out[i] + skew - v * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (d == j) x[j] = 0.f;
    }
  }
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) verify_kernel(VerifyArgs a, DeviceStatus* st) {
  __shared__ int token_s[kMaxNodes], path_s[kMaxNodes], out_s[kMaxNodes];
  __shared__ float p_s[kMaxNodes], q_s[kMaxNodes], u_s[kMaxNodes];
  __shared__ unsigned long long kids_s[kMaxNodes];
  __shared__ double seg_s[2][kWarps], cta_s[2];  // sums of the warps' runs, and of the CTA's, by pass
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / kCluster, rank = (int)cluster_rank();
  if (a.report && blockIdx.x == 0) {
    bool bad = false;
    for (int i = tid; i < a.B * a.T; i += kThreads) {
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

  int node = 0, n_path = 0, n_out = 0, pass = 0;
  double c = 0.0, W = 1.0, total = 0.0;
  bool summed = false;  // whether the last pass's sums are those of the present residual
  // Sums the present residual (c: with q only where c > 0); every thread has the cluster's sum afterwards.
  auto residual = [&]() {
    Residual r;
    const int64_t at = ((int64_t)b * a.T + node) * a.V;
    r.p = a.probs + at;
    r.q = a.draft_probs && c > 0.0 ? a.draft_probs + at : nullptr;
    r.ch = (float)c;
    r.cl = (float)(c - (double)r.ch);
    r.out = out_s;
    r.n_out = n_out;
    r.V = a.V;
    r.skew = (int)(at & 3);
    return r;
  };
  auto sum_pass = [&]() {
    const Residual r = residual();
    const RowRun run = run_of(((int64_t)b * a.T + node) * a.V, a.V, rank * kWarps + warp);
    Sum2 s;
#pragma unroll 4
    for (int64_t v = run.v0 + lane; v < run.v1; v += 32) {
      float x[4], e[4];
      r.at(v, x, e);
#pragma unroll
      for (int j = 0; j < 4; ++j) s.add(x[j], e[j]);
    }
    double d = (double)s.hi + (double)s.lo;
#pragma unroll
    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) seg_s[pass & 1][warp] = d;
    __syncthreads();
    if (tid == 0) {
      double t = 0.0;
      for (int w = 0; w < kWarps; ++w) t += seg_s[pass & 1][w];
      cta_s[pass & 1] = t;
    }
    cluster_sync();  // (and whoever read the buffer two passes ago is done)
    double t = 0.0;
    for (int k = 0; k < kCluster; ++k) t += remote_double(&cta_s[pass & 1], k);
    ++pass;
    summed = true;
    return t;
  };
  if (T > 0) {
    if (tid == 0) path_s[0] = 0;
    n_path = 1;
    unsigned long long kids = kids_s[0];
    while (kids) {
      const int j = __ffsll((long long)kids) - 1;
      kids &= kids - 1;
      double rx;
      bool yes;
      if (a.draft_probs) {
        rx = (double)p_s[j] - c * (double)q_s[j];
        if (!(rx > 0.0)) rx = 0.0;
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
        __syncthreads();  // out_s is read
        n_out = 0;
        summed = false;
        if (tid == 0) path_s[n_path] = j;
        ++n_path;
      } else if (a.draft_probs) {
        c += W;
        W = total = sum_pass();
      } else {
        __syncthreads();  // out_s is read
        if (tid == 0) out_s[n_out] = token_s[j];
        __syncthreads();
        ++n_out;
        W -= rx;
        summed = false;
      }
    }
    if (!summed) total = sum_pass();
    if (!(total > 0.0) && (c > 0.0 || n_out)) {  // nothing is left (p = q to the last bit): the target's own distribution
      c = 0.0;
      n_out = 0;
      total = sum_pass();
    }
  }
  if (rank == 0) {
    __syncthreads();  // path_s is written
    for (int i = tid; i < a.T; i += kThreads) a.path[(int64_t)b * a.T + i] = i < n_path ? path_s[i] : -1;
    if (tid == 0) a.n_path[b] = n_path;
  }
  // ---- the token: the CTA, the warp's run, the vector and the element at which the running sum first exceeds the target
  if (T == 0 || !(total > 0.0)) {
    if (rank == 0 && tid == 0) a.next[b] = -1;
  } else {
    float ul = a.u_last[b];
    ul = ul > 0.f ? fminf(ul, 0.99999994f) : 0.f;  // (a NaN counts as 0)
    const double target = (double)ul * total;
    const int buf = (pass - 1) & 1;
    double before = 0.0;
    int k = 0;  // the last CTA with a share takes what rounding leaves over
    {
      double run = 0.0;
      bool done = false;
      for (int i = 0; i < kCluster; ++i) {
        const double x = remote_double(&cta_s[buf], i);
        if (!done && x > 0.0) {
          k = i;
          before = run;
          done = run + x > target;
        }
        run += x;
      }
    }
    if (k == rank) {
      int w = 0;
      double run = before;
      bool done = false;
      for (int i = 0; i < kWarps; ++i) {
        const double x = seg_s[buf][i];
        if (!done && x > 0.0) {
          w = i;
          before = run;
          done = run + x > target;
        }
        run += x;
      }
      if (warp == w) {
        const Residual r = residual();
        const RowRun rr = run_of(((int64_t)b * a.T + node) * a.V, a.V, rank * kWarps + warp);
        int64_t last = -1, hit = -1;  // the last element with a share so far; the one
        double sum = before;
        for (int64_t v0 = rr.v0; v0 < rr.v1 && hit < 0; v0 += 32) {
          const int64_t v = v0 + lane;
          float x[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
          if (v < rr.v1) r.at(v, x, e);
          double d[4], mine = 0.0;
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = (double)x[j] + (double)e[j], mine += d[j];
          double incl = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const double t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
          }
          double s = sum + (incl - mine);
          int64_t first = -1, end = -1;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s += d[j];
            if (d[j] > 0.0) {
              end = v * 4 - r.skew + j;
              if (first < 0 && s > target) first = end;
            }
          }
          const unsigned has = __ballot_sync(0xffffffffu, first >= 0), any = __ballot_sync(0xffffffffu, end >= 0);
          if (has) hit = __shfl_sync(0xffffffffu, first, __ffs(has) - 1);
          if (any) last = __shfl_sync(0xffffffffu, end, 31 - __clz(any));
          sum += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) a.next[b] = (int32_t)(hit >= 0 ? hit : last);
      }
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
  verify_kernel<<<(unsigned)(B * kCluster), kThreads, 0, s>>>(a, st);
  return cudaGetLastError();
}

}  // namespace msa
