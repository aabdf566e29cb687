// Attention of a tree of drafted tokens over a cache, on the CUDA cores: few rows to a kv
// head (single tokens), and fp32.
//
// out = softmax(q K^T / sqrt(dh)) V over the slots in front of the tree, a node's ancestors
// and itself.  A row is a (node, query head) pair; the rows of a kv head share its keys.
//
// One cluster of S CTAs to (sequence, kv head, block of R rows): the sequence's slots are
// cut into S equal parts, from its length on the device, and the parts' (O, m, l) are
// joined through distributed shared memory, in rank order: no counters, no second launch,
// and results do not depend on timing.  In a CTA the warps take kStep slots in turn; LPS
// lanes share a slot, each with E of its elements (16 bytes, or 8 of an 8-bit cache), so that
// every load is coalesced, and U slots' K and V are in flight together before the first is
// used.  The U x R dot products are summed over their lanes by halving, which leaves one to
// a lane: a step's masks, maxima and exponentials are one instruction each, and the weights
// go back by shuffles.  Each group of LPS lanes keeps its own online softmax.
//
// Bound by latency over a short cache: launch, length, one round trip for K and V, the join
// (one token, 32 heads, 1024 slots: 8.2 us, of which the bytes are 2.5); one row over a large
// one runs at the rate of its loads (64 sequences of 4096, 32 heads, 4.3 GB in 16 bits: 598
// us, 7.2 TB/s; in 8 bits 373 us).  More rows are bound by instructions, some 450 a step of
// 8 slots at 4 rows, and beyond them the tensor cores' kernel takes over; fp32 has none, and
// nothing large runs there.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "tc_common.cuh"

namespace fdllm {

namespace {

constexpr int kNW = 8;
constexpr int kMaxCluster = 16;
constexpr int kWords = FDLLM_MAX_TREE_NODES / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -3.0e38f;  // maximum before the first slot (finite: -inf minus it is -inf)

using f2 = unsigned long long;  // two floats, as the packed instructions take them
__device__ __forceinline__ f2 pack(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// E elements of a cache row, as they are loaded and as pairs of floats.
template <typename C>
struct Vec;
template <>
struct Vec<float> {
  using Raw = float4;
  using Row = float;  // of q and out
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const Raw& r, f2* f) {
    f[0] = pack(r.x, r.y);
    f[1] = pack(r.z, r.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  using Raw = uint4;
  using Row = __nv_bfloat16;
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const Raw& r, f2* f) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
};
template <>
struct Vec<uint8_t> {  // e4m3
  using Raw = uint2;
  using Row = __nv_bfloat16;
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const Raw& r, f2* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t two = (i < 2 ? r.x : r.y) >> (16 * (i & 1));
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
      f[i] = pack(v.x, v.y);
    }
  }
};

// One lane's load into shared memory, asynchronously.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else if constexpr (BYTES == 8)
    asm volatile("cp.async.ca.shared.global.L2::256B [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// a float of another CTA's shared memory
__device__ __forceinline__ float ld_peer(const float* mine, uint32_t rank) {
  uint32_t at;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

template <typename C, int DH, int R>
struct Shape {
  static constexpr bool kFp8 = sizeof(C) == 1;
  static constexpr int E = Vec<C>::E;    // elements of a lane
  static constexpr int LPS = DH / E;     // lanes of a slot
  static constexpr int SPW = 32 / LPS;   // slots of a warp's load
  // One row: K and V go to registers, 8 loads of each in flight (64 sequences of 4096, 16
  // bits: 595 us; through a ring 660).  More rows leave no registers for that: their loads
  // go through a ring in shared memory, several steps ahead (2 rows: 200 us for 240).
  static constexpr bool kRing = R > 1;
  static constexpr int U = !kRing ? 8 : (4 * R <= LPS ? 4 : LPS / R);  // loads of a step
  static constexpr int NV = U * R;       // scores of LPS lanes in a step, at most one a lane
  static constexpr int kDup = LPS / NV;  // lanes with the same score
  static constexpr int kStep = SPW * U;
  static constexpr int LB = sizeof(typename Vec<C>::Raw);
  static constexpr int kStage = 2 * U * 32 * LB;  // bytes: K, V
  static constexpr int kScale = kFp8 ? 2 * 32 * 4 : 0;
  // of a warp 12 KB in flight, 96 KB of a CTA: two CTAs fit an SM
  static constexpr int kDepth = 12 * 1024 / (kStage + kScale);
  // bytes of a warp: the ring, and in its place at the end the warp's O
  static constexpr int kWarp = kRing ? kDepth * (kStage + kScale) : DH * 4;
  static_assert(NV <= LPS && R * DH * 4 <= kWarp, "a warp's O takes the ring's place");
};

template <typename C, int DH, int R>
__global__ void __launch_bounds__(kNW * 32, 2) tree_rows(TreeAttnArgs a) {
  using Vc = Vec<C>;
  using Sh = Shape<C, DH, R>;
  using Raw = typename Vc::Raw;
  using T = typename Vc::Row;
  constexpr bool kFp8 = Sh::kFp8;
  constexpr int E = Sh::E, LPS = Sh::LPS, SPW = Sh::SPW, U = Sh::U, NV = Sh::NV, kDup = Sh::kDup;
  constexpr int kStep = Sh::kStep, LB = Sh::LB, D = Sh::kDepth;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float sm_m[kNW][R], sm_l[kNW][R];
  __shared__ float part_o[R * DH], part_m[R], part_l[R];  // the CTA's, read by its cluster
  __shared__ int par[FDLLM_MAX_TREE_NODES];
  __shared__ uint32_t anc[R][kWords];  // ancestors of each row's node, and itself
  const int g = a.Hq / a.Hkv, rows = a.T * g;
  const int blocks = (rows + R - 1) / R;
  const uint32_t S = cluster_size(), rank = cluster_rank();
  const int blk = blockIdx.x / S;
  const int bh = blk / blocks, r0 = (blk - bh * blocks) * R;
  const int b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPS, d0 = (lane - sub * LPS) * E;
  const float qscale = kLog2e / sqrtf((float)DH);
  tc::griddep_wait();

  const int len = a.cache_len[b], nn = a.n_nodes ? a.n_nodes[b] : a.T;
  if (len < 0 || nn < 0 || nn > a.T || (long long)len + nn > a.N) {
    if (threadIdx.x == 0) set_status(a.status, FDLLM_ERR_BAD_INDEX);
    return;  // the whole cluster does
  }
  if (r0 / g >= nn) return;  // so here
  const int n = len + nn;
  const int per = (int)(((long long)n + S * kStep - 1) / (S * kStep)) * kStep;
  const int lo = min((int)rank * per, n), hi = min(lo + per, n);

  // ---- the ring: a lane copies what it will read itself, so that it waits for its own
  // copies alone.  Lane's score: slot u (of U), row i
  const int sl = lane - sub * LPS;
  const int u_me = sl / (kDup * R), i_me = sl / kDup - u_me * R;
  const size_t head = ((size_t)b * a.Hkv + h) * a.N;
  const C* K = static_cast<const C*>(a.k_cache) + head * DH + d0;
  const C* V = static_cast<const C*>(a.v_cache) + head * DH + d0;
  uint8_t* mine = ring + warp * Sh::kWarp;
  const uint32_t mine_s = tc::smem_u32(mine) + lane * LB;
  float* sc_mine = reinterpret_cast<float*>(mine + D * Sh::kStage) + lane;
  const uint32_t sc_s = tc::smem_u32(sc_mine);
  auto copy = [&](int s0, int st) {
    if (s0 < hi) {
      const uint32_t dst = mine_s + st * Sh::kStage;
      if (s0 + kStep <= n) {
        const size_t at = (size_t)(s0 + sub) * DH;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          copy_async<LB>(dst + u * 32 * LB, K + at + u * SPW * DH);
          copy_async<LB>(dst + (U + u) * 32 * LB, V + at + u * SPW * DH);
        }
      } else {
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
          const size_t at = (size_t)min(s0 + u * SPW + sub, n - 1) * DH;
          copy_async<LB>(dst + u * 32 * LB, K + at);
          copy_async<LB>(dst + (U + u) * 32 * LB, V + at);
        }
      }
      if constexpr (kFp8) {
        const size_t at = head + min(s0 + u_me * SPW + sub, n - 1);
        copy_async<4>(sc_s + st * 256, a.k_scale + at);
        copy_async<4>(sc_s + st * 256 + 128, a.v_scale + at);
      }
    }
    copy_commit();
  };
  const int first = lo + warp * kStep;
  if constexpr (Sh::kRing)
#pragma unroll
    for (int st = 0; st < D; ++st) copy(first + st * kNW * kStep, st);

  f2 q[R][E / 2];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int t = (r0 + i) / g, j = (r0 + i) - t * g;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) q[i][e] = 0ull;
    if (t < nn) {
      const T* at = static_cast<const T*>(a.q) + (((size_t)b * a.T + t) * a.Hq + h * g + j) * DH + d0;
      if constexpr (sizeof(T) == 4)
        Vec<float>::unpack(*reinterpret_cast<const float4*>(at), q[i]);
      else
        Vec<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(at), q[i]);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) q[i][e] = mul2(q[i][e], pack(qscale, qscale));
    }
  }
  if (hi > len) {  // the part reaches into the tree
    if (a.parent)
      for (int t = threadIdx.x; t < nn; t += kNW * 32) par[t] = a.parent[(size_t)b * a.T + t];
    __syncthreads();
    if (threadIdx.x < R) {
      for (int w = 0; w < kWords; ++w) anc[threadIdx.x][w] = 0u;
      int t = (r0 + threadIdx.x) / g;
      while (t >= 0 && t < nn) {
        anc[threadIdx.x][t >> 5] |= 1u << (t & 31);
        int up = a.parent ? par[t] : t - 1;
        if (up < -1 || up >= t) {
          set_status(a.status, FDLLM_ERR_BAD_INDEX);
          up = -1;
        }
        t = up;
      }
    }
    __syncthreads();
  }

  float m = kNone, l = 0.f;  // of row i_me; l: this lane's own weights
  f2 acc[R][E / 2];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int e = 0; e < E / 2; ++e) acc[i][e] = 0ull;
  int st = 0;
#pragma unroll 1
  for (int s0 = first; s0 < hi; s0 += kNW * kStep) {
    const int slot = s0 + u_me * SPW + sub, node = slot - len;
    const uint8_t* at = mine + st * Sh::kStage + lane * LB;
    Raw kr[Sh::kRing ? 1 : U], vr[Sh::kRing ? 1 : U];
    float ksc = 1.f, vsc = 1.f;
    if constexpr (Sh::kRing) {
      copy_wait<D - 1>();
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        kr[u] = __ldcs(reinterpret_cast<const Raw*>(K + (size_t)min(s0 + u * SPW + sub, n - 1) * DH));
#pragma unroll
      for (int u = 0; u < U; ++u)
        vr[u] = __ldcs(reinterpret_cast<const Raw*>(V + (size_t)min(s0 + u * SPW + sub, n - 1) * DH));
      if constexpr (kFp8) {
        ksc = a.k_scale[head + min(slot, n - 1)];
        vsc = a.v_scale[head + min(slot, n - 1)];
      }
    }
    auto k_of = [&](int u) {
      if constexpr (Sh::kRing)
        return *reinterpret_cast<const Raw*>(at + u * 32 * LB);
      else
        return kr[u];
    };
    auto v_of = [&](int u) {
      if constexpr (Sh::kRing)
        return *reinterpret_cast<const Raw*>(at + (U + u) * 32 * LB);
      else
        return vr[u];
    };
    float x[NV];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f2 f[E / 2];
      Vc::unpack(k_of(u), f);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        f2 dot = mul2(q[i][0], f[0]);
#pragma unroll
        for (int e = 1; e < E / 2; ++e) dot = fma2(q[i][e], f[e], dot);
        const float2 y = unpack2(dot);
        x[u * R + i] = y.x + y.y;
      }
    }
    // summed over the slot's lanes: each round gives half of the scores away, until a lane
    // has one
#pragma unroll
    for (int o = LPS / 2, w = NV / 2; o > 0; o >>= 1, w >>= 1) {
      if (w > 0) {
        const bool up = lane & o;
#pragma unroll
        for (int c = 0; c < w; ++c) {
          const float keep = up ? x[c + w] : x[c], gone = up ? x[c] : x[c + w];
          x[c] = keep + __shfl_xor_sync(0xffffffffu, gone, o);
        }
      } else {
        x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
      }
    }
    const bool see =
        slot < hi && (node < 0 || ((anc[i_me][node >> 5] >> (node & 31)) & 1u));
    float y = x[0];
    if constexpr (kFp8) {
      if constexpr (Sh::kRing) {
        ksc = sc_mine[st * 64];
        vsc = sc_mine[st * 64 + 32];
      }
      y *= ksc;
    }
    if (!see) y = -INFINITY;
    float mn = y;
#pragma unroll
    for (int o = kDup * R; o < LPS; o <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mn = fmaxf(mn, m);
    if (__any_sync(0xffffffffu, mn > m)) {
      const float al = ex2(m - mn);
      m = mn;
      l *= al;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float ai = __shfl_sync(0xffffffffu, al, sub * LPS + i * kDup);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) acc[i][e] = mul2(acc[i][e], pack(ai, ai));
      }
    }
    float p = ex2(y - m);
    l += p;
    if constexpr (kFp8) p *= vsc;
    const uint32_t seen = __ballot_sync(0xffffffffu, see);
    auto add = [&](auto all) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        f2 f[E / 2];
        Vc::unpack(v_of(u), f);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int src = sub * LPS + (u * R + i) * kDup;
          const float pi = __shfl_sync(0xffffffffu, p, src);
          if (decltype(all)::value || ((seen >> src) & 1u))  // what is not seen may be NaN
#pragma unroll
            for (int e = 0; e < E / 2; ++e) acc[i][e] = fma2(pack(pi, pi), f[e], acc[i][e]);
        }
      }
    };
    if (seen == 0xffffffffu)
      add(std::true_type{});
    else
      add(std::false_type{});
    if constexpr (Sh::kRing) {
      copy(s0 + D * kNW * kStep, st);
      if (++st == D) st = 0;
    }
  }

  // ---- the groups of a warp, the warps, the cluster
#pragma unroll
  for (int o = kDup * R; o < LPS; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  copy_wait<0>();
  float* o_warp = reinterpret_cast<float*>(mine);  // [R][DH], where the warp's ring was
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float mi = __shfl_sync(0xffffffffu, m, sub * LPS + i * kDup);
    float li = __shfl_sync(0xffffffffu, l, sub * LPS + i * kDup);
    float o8[E];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const float2 v = unpack2(acc[i][e]);
      o8[2 * e] = v.x;
      o8[2 * e + 1] = v.y;
    }
#pragma unroll
    for (int o = LPS; o < 32; o <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, mi, o), l2 = __shfl_xor_sync(0xffffffffu, li, o);
      const float mn = fmaxf(mi, m2), w1 = ex2(mi - mn), w2 = ex2(m2 - mn);
      mi = mn;
      li = li * w1 + l2 * w2;
#pragma unroll
      for (int e = 0; e < E; ++e)
        o8[e] = o8[e] * w1 + __shfl_xor_sync(0xffffffffu, o8[e], o) * w2;
    }
    __syncwarp();  // the other lanes' last reads of the ring
    if (sub == 0) {
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<float4*>(o_warp + i * DH + d0 + e) =
            make_float4(o8[e], o8[e + 1], o8[e + 2], o8[e + 3]);
      if (lane == 0) {
        sm_m[warp][i] = mi;
        sm_l[warp][i] = li;
      }
    }
  }
  __syncthreads();
  T* out = static_cast<T*>(a.out);
  auto put = [&](int x, float v) {
    const int i = x / DH, d = x - i * DH;
    const int t = (r0 + i) / g, j = (r0 + i) - t * g;
    if (t < nn) Store<T>::st(out + (((size_t)b * a.T + t) * a.Hq + h * g + j) * DH + d, v);
  };
  for (int x = threadIdx.x; x < R * DH; x += kNW * 32) {
    const int i = x / DH, d = x - i * DH;
    float M = kNone;
#pragma unroll
    for (int w = 0; w < kNW; ++w) M = fmaxf(M, sm_m[w][i]);
    float num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < kNW; ++w) {
      const float sc = ex2(sm_m[w][i] - M);
      num += reinterpret_cast<const float*>(ring + w * Sh::kWarp)[x] * sc;
      den += sm_l[w][i] * sc;
    }
    if (S == 1) {
      put(x, num / den);
    } else {
      part_o[x] = num;
      if (d == 0) {
        part_m[i] = M;
        part_l[i] = den;
      }
    }
  }
  if (S == 1) return;
  cluster_sync();
  // each CTA joins its share of the outputs; all loads in flight together
  const int share = R * DH / (int)S;  // S is a power of two, at most 16
  if ((int)threadIdx.x < share) {
    const int x = (int)rank * share + threadIdx.x, i = x / DH;
    float pm[kMaxCluster], pl[kMaxCluster], po[kMaxCluster];
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (c < (int)S) {
        pm[c] = ld_peer(&part_m[i], c);
        pl[c] = ld_peer(&part_l[i], c);
        po[c] = ld_peer(&part_o[x], c);
      }
    float M = kNone;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (c < (int)S) M = fmaxf(M, pm[c]);
    float num = 0.f, den = 0.f;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (c < (int)S) {
        const float sc = ex2(pm[c] - M);
        num += po[c] * sc;
        den += pl[c] * sc;
      }
    put(x, num / den);
  }
  cluster_sync();  // nobody leaves while its shared memory is read
}

// Raises a kernel's limits (shared memory, clusters beyond the portable size), once a
// device (a bit of `done`; setting them twice does no harm).
cudaError_t allow(const void* kern, int smem, std::atomic<unsigned long long>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}
template <typename C, int DH, int R>
std::atomic<unsigned long long> allowed{0};

template <typename C, int DH, int R>
cudaError_t launch(const TreeAttnArgs& a, cudaStream_t stream) {
  using Sh = Shape<C, DH, R>;
  constexpr int kSmem = kNW * Sh::kWarp;
  const int rows = a.T * (a.Hq / a.Hkv);
  const long long blocks = (long long)a.B * a.Hkv * ((rows + R - 1) / R);
  // Parts of a sequence: as many as two CTAs to an SM take (more CTAs, for fuller waves,
  // cost more than the waves: 121 us for 36 at 64 blocks cut into 16 parts for 4).  Nothing
  // here depends on the cache's capacity: the same tokens give the same bits in any.
  const int most = 2 * device_sm_count();
  int S = 1;
  while (S < kMaxCluster && blocks * S * 2 <= most) S *= 2;
  auto kern = tree_rows<C, DH, R>;
  const cudaError_t err = allow(reinterpret_cast<const void*>(kern), kSmem, &allowed<C, DH, R>);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks * S));
  cfg.blockDim = dim3(kNW * 32);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  count_launches(1);
  return e;
}
template <typename C>
cudaError_t launch_c(const TreeAttnArgs& a, cudaStream_t stream) {
  const int rows = a.T * (a.Hq / a.Hkv);
  if (rows == 1) return a.dh == 64 ? launch<C, 64, 1>(a, stream) : launch<C, 128, 1>(a, stream);
  if constexpr (sizeof(C) < 4)
    if (rows == 2) return a.dh == 64 ? launch<C, 64, 2>(a, stream) : launch<C, 128, 2>(a, stream);
  return a.dh == 64 ? launch<C, 64, 4>(a, stream) : launch<C, 128, 4>(a, stream);
}

}  // namespace

// fp32; one row to a kv head, whatever the size (one sequence of 1024, 32 kv heads: 8.2 us,
// on the tensor cores 21.9; 64 of 4096: 598 for 650 in 16 bits, 373 for 573 in 8); up to 4
// rows where the sequences' kv heads are few, so that latency counts (4 rows, 8 kv heads, 16
// and 8 bits: 1 x 1024 12.3 for 16.4 and 12.3 for 20.5, 8 x 4096 38.9 for 36.5 and 40.5 for
// 41.0).  The lengths are on the device, so that the rule cannot know them: 8 of 16384 lose
// by it (100.7 for 96.2, 109.9 for 86.1).  With more heads the instructions of 4 rows cost
// more than the tensor cores' kernel takes (64 x 4096: 186 for 176, 208 for 160; 2 rows of 16
// bits 195 for 175, of 8 bits 155 for 159).
bool tree_simt_takes(const TreeAttnArgs& a) {
  const int rows = a.T * (a.Hq / a.Hkv);
  return a.dtype == FDLLM_F32 || rows == 1 || (rows <= 4 && a.B * a.Hkv <= 64);
}

cudaError_t launch_tree_simt(const TreeAttnArgs& a, cudaStream_t stream) {
  if (a.dtype == FDLLM_F32) return launch_c<float>(a, stream);
  return a.fp8 ? launch_c<uint8_t>(a, stream) : launch_c<__nv_bfloat16>(a, stream);
}

}  // namespace fdllm
