// Rows of k and v in 8 bits: quantised as they are written into a cache, and
// read back.
//
// Mathematics, per row x[dh] of one head: a = max |x| within [2^-96, FLT_MAX],
// scale = a / 448, element = e4m3(x * (448 / a)); 448 is e4m3's largest value,
// so the row's largest element uses the whole range.  The bounds on a keep
// 448 / a finite and normal for rows of zeros, denormals and infinities.  The
// two quotients are IEEE divisions and the product is rounded once in fp32, so
// that the stored bits do not depend on the kernel's shape.
//
// Bound: HBM.  A row-head moves dh * (2 + 1) + 4 bytes (bf16).  A group of dh/8
// lanes owns one row-head and holds 8 elements of k and 8 of v a lane, so that a
// warp has 16-byte loads of 4 head rows in flight, the maximum is 3 or 4
// shuffles and every store is 8 contiguous bytes a lane.
//
// A CTA takes a block of rows of one sequence.  Rows of the same slot: the
// highest index is kept.  The CTA reads the positions behind its block once and
// marks the rows that a later one replaces; blocks are larger where a sequence
// has many rows, so that this scan stays small beside the rows themselves.
#include <float.h>

#include "common.cuh"
#include "kernels.h"

namespace fdllm {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlockRows = 16;
constexpr float kFp8Max = 448.f;
constexpr float kTiny = 1.262177448353618888e-29f;  // 2^-96

// two floats to e4m3 (nearest even, beyond 448 to 448, NaN stays NaN): lo in the
// low byte
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

// Quantises 8 elements a lane of a row held by G lanes; returns the row's scale.
template <int G>
__device__ __forceinline__ float quantise8(const float* x, uint2* q) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));  // leaves a NaN out
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  a = fminf(fmaxf(a, kTiny), FLT_MAX);
  const float inv = __fdiv_rn(kFp8Max, a);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(x[i], inv);
  q->x = e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16);
  q->y = e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16);
  return __fdiv_rn(a, kFp8Max);
}

// grid B * blocks; a CTA's units are the (row, head) pairs of its block of rows.
template <typename T, int DH>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(CacheFp8Args a, int block_rows,
                                                               int blocks) {
  constexpr int G = DH / 8;  // lanes of a row-head
  constexpr int kGroups = kThreads / G;
  __shared__ int s_pos[kMaxBlockRows];
  const int b = blockIdx.x / blocks, r0 = (blockIdx.x - b * blocks) * block_rows;
  const int nr = min(block_rows, a.R - r0);
  const int32_t* pos = a.pos + (size_t)b * a.R;
  const int tid = threadIdx.x;
  if (tid < nr) {
    const int p = pos[r0 + tid];
    if (p < -1 || p >= a.N) set_status(a.status, FDLLM_ERR_BAD_INDEX);
    s_pos[tid] = p >= a.N ? -1 : p;
  }
  if (r0 + 1 < a.R) {  // a later row of the same slot replaces this block's
    __syncthreads();
    int mine[kMaxBlockRows];
#pragma unroll
    for (int i = 0; i < kMaxBlockRows; ++i) mine[i] = i < nr ? s_pos[i] : -1;
    __syncthreads();
    for (int j = r0 + 1 + tid; j < a.R; j += kThreads) {
      const int p = pos[j];
#pragma unroll
      for (int i = 0; i < kMaxBlockRows; ++i)
        if (p == mine[i] && j > r0 + i) s_pos[i] = -1;
    }
  }
  __syncthreads();

  const int g = tid / G, gl = tid % G;
  const int units = nr * a.H;
  const size_t head0 = (size_t)b * a.H;
  // whole warps go through the loop together: the shuffles need every lane
  for (int u0 = 0; u0 < units; u0 += kGroups) {
    const int u = u0 + g;
    const bool in = u < units;
    const int row = in ? u / a.H : 0, h = in ? u - row * a.H : 0;
    const int p = in ? s_pos[row] : -1;
    float k[8], v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = v[i] = 0.f;
    if (p >= 0) {
      const size_t src = (((size_t)b * a.R + r0 + row) * a.H + h) * DH + gl * 8;
      load8(static_cast<const T*>(a.k_rows) + src, k);
      load8(static_cast<const T*>(a.v_rows) + src, v);
    }
    uint2 kq, vq;
    const float ks = quantise8<G>(k, &kq);
    const float vs = quantise8<G>(v, &vq);
    if (p >= 0) {
      const size_t slot = (head0 + h) * a.N + p;
      *reinterpret_cast<uint2*>(a.k_cache + slot * DH + gl * 8) = kq;
      *reinterpret_cast<uint2*>(a.v_cache + slot * DH + gl * 8) = vq;
      if (gl == 0) {
        a.k_scale[slot] = ks;
        a.v_scale[slot] = vs;
      }
    }
  }
}

// grid B * blocks, as the write.
template <typename T, int DH>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheFp8Args a, int block_rows,
                                                              int blocks) {
  constexpr int G = DH / 8;
  constexpr int kGroups = kThreads / G;
  const int b = blockIdx.x / blocks, r0 = (blockIdx.x - b * blocks) * block_rows;
  const int nr = min(block_rows, a.R - r0);
  const int32_t* pos = a.pos + (size_t)b * a.R;
  const int tid = threadIdx.x;
  const int g = tid / G, gl = tid % G;
  const size_t head0 = (size_t)b * a.H;
  for (int u = g; u < nr * a.H; u += kGroups) {
    // head after head, rows innermost: neighbouring groups read neighbouring slots
    const int h = u / nr, row = u - h * nr;
    const int p = pos[r0 + row];
    if (p < 0 || p >= a.N) {
      if (p != -1 && h == 0 && gl == 0) set_status(a.status, FDLLM_ERR_BAD_INDEX);
      continue;
    }
    const size_t slot = (head0 + h) * a.N + p;
    const uint2 kq = __ldcs(reinterpret_cast<const uint2*>(a.k_cache + slot * DH + gl * 8));
    const uint2 vq = __ldcs(reinterpret_cast<const uint2*>(a.v_cache + slot * DH + gl * 8));
    const float ks = a.k_scale[slot], vs = a.v_scale[slot];
    float k[8], v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t kw = i < 2 ? kq.x : kq.y, vw = i < 2 ? vq.x : vq.y;
      const float2 kf = from_e4m3x2((i & 1) ? kw >> 16 : kw & 0xffffu);
      const float2 vf = from_e4m3x2((i & 1) ? vw >> 16 : vw & 0xffffu);
      k[2 * i] = kf.x * ks;
      k[2 * i + 1] = kf.y * ks;
      v[2 * i] = vf.x * vs;
      v[2 * i + 1] = vf.y * vs;
    }
    const size_t dst = (((size_t)b * a.R + r0 + row) * a.H + h) * DH + gl * 8;
    store8(static_cast<T*>(a.k_rows) + dst, k);
    store8(static_cast<T*>(a.v_rows) + dst, v);
  }
}

// Rows of a CTA's block: enough (row, head) pairs for two rounds of its groups,
// and 16 where a sequence's rows are so many that the scan for replaced rows
// would otherwise be read too often.
int rows_per_block(const CacheFp8Args& a) {
  if (a.R > 1024) return kMaxBlockRows;
  const int groups = kThreads / (a.dh / 8);
  int n = (2 * groups + a.H - 1) / a.H;
  return n > kMaxBlockRows ? kMaxBlockRows : n;
}

template <typename T, int DH>
cudaError_t launch(const CacheFp8Args& a, bool write, cudaStream_t stream) {
  const int n = rows_per_block(a);
  const int blocks = (a.R + n - 1) / n;
  if (write)
    cache_write_kernel<T, DH><<<a.B * blocks, kThreads, 0, stream>>>(a, n, blocks);
  else
    cache_read_kernel<T, DH><<<a.B * blocks, kThreads, 0, stream>>>(a, n, blocks);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t dispatch(const CacheFp8Args& a, bool write, cudaStream_t stream) {
  if (a.dtype == FDLLM_F32)
    return a.dh == 64 ? launch<float, 64>(a, write, stream) : launch<float, 128>(a, write, stream);
  return a.dh == 64 ? launch<__nv_bfloat16, 64>(a, write, stream)
                    : launch<__nv_bfloat16, 128>(a, write, stream);
}

}  // namespace

cudaError_t launch_cache_write_fp8(const CacheFp8Args& a, cudaStream_t stream) {
  return dispatch(a, true, stream);
}
cudaError_t launch_cache_read_fp8(const CacheFp8Args& a, cudaStream_t stream) {
  return dispatch(a, false, stream);
}

}  // namespace fdllm
