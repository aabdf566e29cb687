// Attention of a tree of drafted tokens over an fp32 cache, on the CUDA cores.
//
// out = softmax(q K^T / sqrt(dh)) V over the slots in front of the tree, a node's
// ancestors and itself; query heads share kv heads in groups of g = Hq / Hkv.
//
// One CTA (8 warps) per (sequence, kv head, group of 4 query rows), a row being a
// (node, query head) pair.  Warps take keys round-robin; the lanes of a warp split
// the head dimension, so each key row is one coalesced load.  Each warp keeps an
// online softmax per row; the warps are merged at the end.  Bound by the
// instructions of the per-key reductions; it serves fp32 storage, where nothing
// large runs.
#include "common.cuh"
#include "kernels.h"

namespace fdllm {

namespace {

constexpr int kQG = 4;
constexpr int kNW = 8;
constexpr int kWords = FDLLM_MAX_TREE_NODES / 32;
constexpr float kLog2e = 1.4426950408889634f;

template <int EPL>
__global__ void __launch_bounds__(kNW * 32) tree_simt(TreeAttnArgs a) {
  constexpr int dh = EPL * 32;
  __shared__ float sm_m[kNW][kQG], sm_l[kNW][kQG];
  __shared__ float sm_acc[kNW][kQG][dh];
  __shared__ uint32_t anc[kQG][kWords];  // ancestors of each row's node, and itself
  const int g = a.Hq / a.Hkv, rows = a.T * g;
  const int blocks = (rows + kQG - 1) / kQG;
  const int bh = blockIdx.x / blocks, r0 = (blockIdx.x - bh * blocks) * kQG;
  const int b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float qscale = kLog2e / sqrtf((float)dh);

  const int len = a.cache_len[b], nn = a.n_nodes ? a.n_nodes[b] : a.T;
  if (len < 0 || nn < 0 || nn > a.T || (long long)len + nn > a.N) {
    if (threadIdx.x == 0) set_status(a.status, FDLLM_ERR_BAD_INDEX);
    return;
  }
  const int32_t* parent = a.parent ? a.parent + (size_t)b * a.T : nullptr;
  if (threadIdx.x < kQG) {
    const int t = (r0 + threadIdx.x) / g;
    for (int w = 0; w < kWords; ++w) anc[threadIdx.x][w] = 0u;
    if (t < nn) {
      for (int n = t; n >= 0;) {
        anc[threadIdx.x][n >> 5] |= 1u << (n & 31);
        int par = parent ? parent[n] : n - 1;
        if (par < -1 || par >= n) {
          set_status(a.status, FDLLM_ERR_BAD_INDEX);
          par = -1;
        }
        n = par;
      }
    }
  }
  __syncthreads();

  float q[kQG][EPL];
  bool used[kQG];
#pragma unroll
  for (int i = 0; i < kQG; ++i) {
    const int t = (r0 + i) / g, j = (r0 + i) - t * g;
    used[i] = t < nn;
#pragma unroll
    for (int e = 0; e < EPL; ++e)
      q[i][e] = used[i] ? qscale * static_cast<const float*>(
                                       a.q)[(((size_t)b * a.T + t) * a.Hq + h * g + j) * dh +
                                            lane * EPL + e]
                        : 0.f;
  }
  float m[kQG], l[kQG], acc[kQG][EPL];
#pragma unroll
  for (int i = 0; i < kQG; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[i][e] = 0.f;
  }
  const size_t head = ((size_t)b * a.Hkv + h) * a.N;
  const float* K = static_cast<const float*>(a.k_cache) + head * dh + lane * EPL;
  const float* V = static_cast<const float*>(a.v_cache) + head * dh + lane * EPL;
  for (int s = warp; s < len + nn; s += kNW) {
    bool see[kQG];
    bool any = false;
#pragma unroll
    for (int i = 0; i < kQG; ++i) {
      const int j = s - len;
      see[i] = used[i] && (j < 0 || ((anc[i][j >> 5] >> (j & 31)) & 1u));
      any |= see[i];
    }
    if (!any) continue;
    float k[EPL], v[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      k[e] = K[(size_t)s * dh + e];
      v[e] = V[(size_t)s * dh + e];
    }
#pragma unroll
    for (int i = 0; i < kQG; ++i) {
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) x = fmaf(q[i][e], k[e], x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (!see[i]) continue;
      const float mn = fmaxf(m[i], x);
      const float sc = (m[i] == -INFINITY) ? 0.f : exp2f(m[i] - mn);
      const float p = x == -INFINITY ? 0.f : exp2f(x - mn);  // not 2^(-inf + inf)
      l[i] = l[i] * sc + p;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[i][e] = fmaf(p, v[e], acc[i][e] * sc);
      m[i] = mn;
    }
  }
#pragma unroll
  for (int i = 0; i < kQG; ++i) {
    if (lane == 0) {
      sm_m[warp][i] = m[i];
      sm_l[warp][i] = l[i];
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) sm_acc[warp][i][lane * EPL + e] = acc[i][e];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < kQG * dh; x += blockDim.x) {
    const int i = x / dh, d = x - i * dh;
    const int t = (r0 + i) / g, j = (r0 + i) - t * g;
    if (t >= nn) continue;
    float M = -INFINITY;
    for (int w = 0; w < kNW; ++w) M = fmaxf(M, sm_m[w][i]);
    float num = 0.f, den = 0.f;
    for (int w = 0; w < kNW; ++w) {
      const float sc = (sm_m[w][i] == -INFINITY) ? 0.f : exp2f(sm_m[w][i] - M);
      num += sm_acc[w][i][d] * sc;
      den += sm_l[w][i] * sc;
    }
    static_cast<float*>(a.out)[(((size_t)b * a.T + t) * a.Hq + h * g + j) * dh + d] = num / den;
  }
}

}  // namespace

cudaError_t launch_tree_simt(const TreeAttnArgs& a, cudaStream_t stream) {
  const int rows = a.T * (a.Hq / a.Hkv);
  const int grid = a.B * a.Hkv * ((rows + kQG - 1) / kQG);
  if (a.dh == 64)
    tree_simt<2><<<grid, kNW * 32, 0, stream>>>(a);
  else
    tree_simt<4><<<grid, kNW * 32, 0, stream>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace fdllm
