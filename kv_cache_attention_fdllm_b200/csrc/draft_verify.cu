// Verification of drafted tokens against the target's probabilities from given
// random numbers: a chain of sampled drafts, or a tree of candidates.
//
// Mathematics.  Chain: draft x ~ q is accepted iff u q(x) < p(x); after the first
// that is not, the next token is drawn from max(p - q, 0), which together leaves
// every token distributed as p.  Tree: a node's children were not sampled; one
// number u picks the first child whose running sum of p exceeds it, and without
// one the next token is drawn from p without the children, which again is p.
// A draw from weights w is the smallest v with cumsum(w)_v > r sum(w).
//
// All of it in 64 bits: a product of two floats is exact in fp64, and sums over a
// vocabulary are off by some 1e-15, so that the tokens do not depend on how the
// sums are split.  (fp32 sums are off by 1e-7 of the total, while the steps of a
// cumsum over 126464 tokens are 1e-5 wide on average: one draw in a hundred would
// give another token.)
//
// Bound: HBM over one row pair (tree: one row) a sequence, and latency below some
// tens of sequences.  One launch: every CTA of a sequence walks its drafts itself
// (all gathers at once, then shared memory), which costs less than a second
// launch; its warps then sum sub-blocks of 512 weights, 16-byte loads all in
// flight before the first is used; the last CTA of the sequence to finish finds
// the sub-block that holds r sum(w) from the sums, and in it the token.  Measured at a
// vocabulary of 126464: 8 chains of 5 drafts 8.2 us, 64 of 4 16.4-18.0 us (64.8 MB; the more
// the less of them L2 holds), 8 trees of 40 nodes 10.3 us; of the 8.2 us the walk takes 1.5, the sums 2.6, the count 1, the draw
// 2.8, each a dependent round trip or two.
#include <limits.h>

#include "common.cuh"
#include "kernels.h"

namespace fdllm {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSub = 512;  // weights of one partial sum: 4 x 4 a lane
constexpr int kMaxNodes = FDLLM_MAX_TREE_NODES;

// A child's tokens are left out of a tree's draw: at most kMaxNodes - 1 of them.
struct Weights {
  const float* p;
  const float* q;  // null: weights are p
  int V;
  bool vec;        // rows start on 16-byte boundaries
};

__device__ __forceinline__ double weight(float p, float q) {
  return fmax((double)p - (double)q, 0.0);  // a NaN gives 0
}

// w[0..3] of the weights at i .. i+3 (0 behind V)
__device__ __forceinline__ void load4(const Weights& w, int i, float4* p, float4* q) {
  *p = make_float4(0.f, 0.f, 0.f, 0.f);
  *q = *p;
  if (w.vec && i + 3 < w.V) {
    *p = __ldg(reinterpret_cast<const float4*>(w.p + i));
    if (w.q) *q = __ldg(reinterpret_cast<const float4*>(w.q + i));
  } else {
    float pv[4], qv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      pv[e] = i + e < w.V ? __ldg(w.p + i + e) : 0.f;
      qv[e] = w.q && i + e < w.V ? __ldg(w.q + i + e) : 0.f;
    }
    *p = make_float4(pv[0], pv[1], pv[2], pv[3]);
    *q = make_float4(qv[0], qv[1], qv[2], qv[3]);
  }
}

// Sets the weights at i .. i+3 of a listed token to 0.
__device__ __forceinline__ void leave_out(const int* out, int n_out, int i, float4* p) {
  for (int k = 0; k < n_out; ++k) {
    const int e = out[k] - i;
    if (e == 0) p->x = 0.f;
    if (e == 1) p->y = 0.f;
    if (e == 2) p->z = 0.f;
    if (e == 3) p->w = 0.f;
  }
}

__device__ __forceinline__ double sum4(const float4& p, const float4& q) {
  return (weight(p.x, q.x) + weight(p.y, q.y)) + (weight(p.z, q.z) + weight(p.w, q.w));
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum of sub-block s by one warp.
__device__ __forceinline__ double sub_sum(const Weights& w, int s, const int* out, int n_out,
                                          int lane) {
  const int i0 = s * kSub + lane * 4;
  float4 p[4], q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) load4(w, i0 + k * 128, &p[k], &q[k]);
  if (n_out) {
#pragma unroll
    for (int k = 0; k < 4; ++k) leave_out(out, n_out, i0 + k * 128, &p[k]);
  }
  double t = 0.0;
#pragma unroll
  for (int k = 0; k < 4; ++k) t += sum4(p[k], q[k]);
  return warp_sum(t);
}

struct Scan {
  double warp[kWarps];
};
// Inclusive sum over the CTA's threads in order, and the CTA's total.
__device__ __forceinline__ double block_scan(double v, Scan& sh, double* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  __syncthreads();  // the last use of sh is over
  if (lane == 31) sh.warp[warp] = v;
  __syncthreads();
  double base = 0.0, all = 0.0;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    if (k < warp) base += sh.warp[k];
    all += sh.warp[k];
  }
  *total = all;
  return base + v;
}

struct Pick {
  int best;        // candidate index, INT_MAX for none
  int last;        // last index with a positive weight, -1 for none
  double base;     // sum in front of the sub-block
};

// The token drawn from w by r, whose sub-block sums are parts[0..n_sub) (read
// around L1: other CTAs wrote them).  Whole CTA; every thread gets the result,
// -1 where every weight is 0.
__device__ int draw(const Weights& w, const double* parts, int n_sub, float r, const int* out,
                    int n_out, Scan& sh, Pick& pk) {
  const int tid = threadIdx.x;
  const double rr = (double)fminf(fmaxf(r, 0.f), 0.99999994f);
  // the running sums (of the one round of threads that a vocabulary usually needs, kept)
  double total = 0.0, x = 0.0, c = 0.0;
  for (int s0 = 0; s0 < n_sub; s0 += kThreads) {
    x = s0 + tid < n_sub ? __ldcg(parts + s0 + tid) : 0.0;
    double t;
    c = total + block_scan(x, sh, &t);
    total += t;
  }
  if (!(total > 0.0)) return -1;
  const double want = rr * total;
  // the first sub-block whose running sum exceeds it; the last with any weight
  // where rounding leaves none
  if (tid == 0) {
    pk.best = INT_MAX;
    pk.last = -1;
    pk.base = 0.0;
  }
  __syncthreads();
  double base = 0.0;
  for (int s0 = 0; s0 < n_sub; s0 += kThreads) {
    if (n_sub > kThreads) {
      x = s0 + tid < n_sub ? __ldcg(parts + s0 + tid) : 0.0;
      double t;
      c = base + block_scan(x, sh, &t);
      base += t;
    }
    if (x > 0.0 && c > want) atomicMin(&pk.best, s0 + tid);
    if (x > 0.0) atomicMax(&pk.last, s0 + tid);
    __syncthreads();
    if (pk.best == s0 + tid || (pk.best == INT_MAX && pk.last == s0 + tid)) pk.base = c - x;
    __syncthreads();
    if (pk.best != INT_MAX) break;
  }
  const int sub = pk.best != INT_MAX ? pk.best : pk.last;
  base = pk.base;
  __syncthreads();
  if (tid == 0) {
    pk.best = INT_MAX;
    pk.last = -1;
  }
  // its weights, 2 a thread in order
  static_assert(kSub == 2 * kThreads, "two weights a thread");
  const int i = sub * kSub + tid * 2;
  double y[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float p = i + e < w.V ? __ldg(w.p + i + e) : 0.f;
    const float q = w.q && i + e < w.V ? __ldg(w.q + i + e) : 0.f;
    for (int k = 0; k < n_out; ++k)
      if (out[k] == i + e) p = 0.f;
    y[e] = weight(p, q);
  }
  double t;
  c = base + block_scan(y[0] + y[1], sh, &t) - (y[0] + y[1]);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    c += y[e];
    if (y[e] > 0.0) {
      if (c > want) atomicMin(&pk.best, i + e);
      atomicMax(&pk.last, i + e);
    }
  }
  __syncthreads();
  return pk.best != INT_MAX ? pk.best : pk.last;
}

// grid B * ctas: `ctas` CTAs a sequence
template <bool TREE>
__global__ void __launch_bounds__(kThreads, 4) draft_verify_kernel(DraftVerifyArgs a, int ctas) {
  const int b = blockIdx.x / ctas, cta = blockIdx.x - b * ctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int T = a.T, V = a.V;
  const bool first_cta = cta == 0;
  const int32_t* tok = a.tok + (size_t)b * T;
  const float* u = a.u + (size_t)b * T;
  int n = a.count ? a.count[b] : T;
  const int n_lo = TREE ? 1 : 0;
  if (n < n_lo || n > T) {
    if (first_cta && tid == 0) set_status(a.status, FDLLM_ERR_BAD_INDEX);
    n = n < n_lo ? n_lo : T;
  }

  __shared__ int s_out[TREE ? kMaxNodes : 1];  // the final node's children's tokens
  __shared__ int s_n_out, s_node, s_len, s_last;
  __shared__ Scan s_scan;
  __shared__ Pick s_pick;
  if (tid == 0) s_n_out = 0;

  // ---- the walk
  if constexpr (TREE) {
    __shared__ int s_par[kMaxNodes], s_tok[kMaxNodes], s_path[kMaxNodes];
    __shared__ float s_w[kMaxNodes], s_u[kMaxNodes];
    static_assert(kMaxNodes <= kThreads, "one thread a node");
    int par = -1, tk = 0;
    if (tid < n) {
      s_u[tid] = u[tid];
      if (tid > 0) {
        par = a.parent[(size_t)b * T + tid];
        tk = tok[tid];
        if (par < 0 || par >= tid || tk < 0 || tk >= V) {
          if (first_cta) set_status(a.status, FDLLM_ERR_BAD_INDEX);
          par = -1;  // never reached
        } else {
          s_w[tid] = a.target[((size_t)b * T + par) * V + tk];
        }
      }
      s_tok[tid] = tk;
    }
    if (tid < kMaxNodes) s_par[tid] = par;
    __syncthreads();
    if (warp == 0) {
      // one warp walks: the children of the node are a ballot over 32 nodes at a time,
      // taken in order until the running sum exceeds the node's number
      int node = 0, len = 0;
      for (int next = 0; next >= 0;) {
        const double un = (double)s_u[node];
        double c = 0.0;
        next = -1;
        for (int k = 0; k < n && next < 0; k += 32) {
          unsigned kids = __ballot_sync(0xffffffffu, s_par[k + lane] == node);
          while (kids && next < 0) {
            const int j = k + __ffs(kids) - 1;
            c += fmax((double)s_w[j], 0.0);
            if (un < c) next = j;
            // siblings behind it that repeat its token add nothing: out of the tree
            const int x = s_tok[j];
            __syncwarp();
            for (int m = k; m < n; m += 32) {
              const int t = m + lane;
              if (t > j && s_par[t] == node && s_tok[t] == x) s_par[t] = -1;
            }
            __syncwarp();
            kids = __ballot_sync(0xffffffffu, s_par[k + lane] == node && k + lane > j);
          }
        }
        if (next >= 0) {
          if (lane == 0) s_path[len] = next;
          ++len;
          node = next;
        }
      }
      if (lane == 0) {
        s_node = node;
        s_len = len;
      }
    }
    __syncthreads();
    if (par == s_node) s_out[atomicAdd(&s_n_out, 1)] = tk;
    if (first_cta)
      for (int t = tid; t < T; t += kThreads)
        a.path[(size_t)b * T + t] = t < s_len ? s_path[t] : -1;
  } else {
    if (tid == 0) s_node = n;
    __syncthreads();
    for (int t = tid; t < n; t += kThreads) {
      const int x = tok[t];
      bool take = false;
      if (x < 0 || x >= V) {
        if (first_cta) set_status(a.status, FDLLM_ERR_BAD_INDEX);
      } else {
        const float p = a.target[((size_t)b * (T + 1) + t) * V + x];
        const float q = a.draft[((size_t)b * T + t) * V + x];
        take = (double)u[t] * (double)q < (double)p;  // exact; a NaN is not accepted
      }
      if (!take) atomicMin(&s_node, t);
    }
    __syncthreads();
    if (tid == 0) s_len = s_node;
  }
  __syncthreads();

  // ---- the weights of the draw, summed by sub-blocks
  const int node = s_node, n_out = TREE ? s_n_out : 0;
  Weights w;
  w.V = V;
  w.p = a.target + ((size_t)b * (TREE ? T : T + 1) + node) * V;
  w.q = !TREE && node < n ? a.draft + ((size_t)b * T + node) * V : nullptr;
  w.vec = ((reinterpret_cast<uintptr_t>(w.p) | reinterpret_cast<uintptr_t>(w.q)) & 15u) == 0;
  const int n_sub = (V + kSub - 1) / kSub;
  double* parts = a.parts + (size_t)b * n_sub;
  for (int s = cta * kWarps + warp; s < n_sub; s += ctas * kWarps) {
    const double t = sub_sum(w, s, s_out, n_out, lane);
    if (lane == 0) __stcg(parts + s, t);
  }
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(&a.seq_cnt[b], 1u) == (unsigned)ctas - 1u;
    if (s_last) {
      __threadfence();
      a.seq_cnt[b] = 0u;  // for the next call
    }
  }
  __syncthreads();
  if (!s_last) return;

  // ---- the last CTA of the sequence draws
  const float r = a.r[b];
  int v = draw(w, parts, n_sub, r, s_out, n_out, s_scan, s_pick);
  if (v < 0 && (w.q || n_out)) {
    // no weight is left: the target's own row
    w.q = nullptr;
    w.vec = (reinterpret_cast<uintptr_t>(w.p) & 15u) == 0;
    __syncthreads();
    for (int s = warp; s < n_sub; s += kWarps) {
      const double t = sub_sum(w, s, s_out, 0, lane);
      if (lane == 0) __stcg(parts + s, t);
    }
    __syncthreads();
    v = draw(w, parts, n_sub, r, s_out, 0, s_scan, s_pick);
  }
  if (tid == 0) {
    a.next_tok[b] = v;
    a.n_accept[b] = s_len;
  }
}

// CTAs of a sequence: four a SM over all of them, which is what is resident (one CTA more
// a sequence and the last start when the first end: 20.6 us for 17.8, measured together, for
// 64 chains of 4 drafts over 126464 tokens), no more than one round of sub-blocks each.
int ctas_per_seq(int B, int V) {
  const int n_sub = (V + kSub - 1) / kSub;
  const int most = (n_sub + kWarps - 1) / kWarps;
  int n = 4 * device_sm_count() / B;
  return n < 1 ? 1 : (n > most ? most : n);
}

}  // namespace

size_t draft_verify_parts_bytes(int B, int V) {
  return align_up((size_t)B * (((size_t)V + kSub - 1) / kSub) * sizeof(double), 256);
}

cudaError_t launch_chain_verify(const DraftVerifyArgs& a, cudaStream_t stream) {
  const int n = ctas_per_seq(a.B, a.V);
  draft_verify_kernel<false><<<a.B * n, kThreads, 0, stream>>>(a, n);
  count_launches(1);
  return cudaGetLastError();
}
cudaError_t launch_tree_verify(const DraftVerifyArgs& a, cudaStream_t stream) {
  const int n = ctas_per_seq(a.B, a.V);
  draft_verify_kernel<true><<<a.B * n, kThreads, 0, stream>>>(a, n);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace fdllm
