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
// Bound: HBM, closely followed by the instructions of the write (maxima, quotients,
// conversions).  A row-head moves dh * (2 + 1) + 4 bytes (bf16).  A group of dh/8 lanes
// owns one row-head of k and of v, 8 elements a lane, and has two of each in flight; the
// maxima of bf16 rows are taken as whole numbers, two at a time, those of k in the even
// lanes and of v in the odd ones, so that a lane divides once for its row and the maximum
// costs 3 or 4 shuffles for both.  Measured: 64 x 500 rows of 8 heads of 128, 199 MB:
// 43 us, 4.6 TB/s (57 us with plain maxima and two quotients a lane and row); 16384 slots
// of 32 heads read back, 407 MB: 76 us, 5.3 TB/s.
//
// A CTA takes a block of rows of one sequence.  Rows of the same slot: the
// highest index is kept.  The CTA reads the positions behind its block once and
// marks the rows that a later one replaces; blocks are larger where a sequence
// has many rows, so that this scan stays small beside the rows themselves.
#include <float.h>
#include <limits.h>

#include "common.cuh"
#include "kernels.h"

namespace fdllm {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlockRows = 16;
constexpr int kUnits = 2;  // (row, head) units of a group in flight, write
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

// 8 elements of a row as they are loaded
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  // largest |x| but for NaN
  __device__ __forceinline__ float top() const {
    return fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                 fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  // largest |x|, two at a time: magnitudes compare as whole numbers, a NaN above them all
  // (then one by one, without it)
  __device__ __forceinline__ float top() const {
    const uint32_t m = __vmaxu2(__vmaxu2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu),
                                __vmaxu2(a.z & 0x7fff7fffu, a.w & 0x7fff7fffu));
    uint32_t t = max(m & 0xffffu, m >> 16);
    if (t > 0x7f80u) {
      t = 0u;
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t e = (w[i >> 1] >> (16 * (i & 1))) & 0x7fffu;
        if (e <= 0x7f80u) t = max(t, e);
      }
    }
    return __uint_as_float(t << 16);
  }
};
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

__device__ __forceinline__ uint2 quantise8(const float* x, float inv) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(x[i], inv);
  return make_uint2(e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16),
                    e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16));
}

// 8 elements of a row and its scale as floats
__device__ __forceinline__ void dequantise8(uint2 q, float scale, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? q.x : q.y;
    const float2 f = from_e4m3x2((i & 1) ? w >> 16 : w & 0xffffu);
    v[2 * i] = f.x * scale;
    v[2 * i + 1] = f.y * scale;
  }
}

// grid B * blocks; a CTA's units are the (row, head) pairs of its block of rows.  A group
// has the rows of two units in flight; the first two are loaded before the positions are
// looked at, whose latencies then lie beside theirs.
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
  const int g = tid / G, gl = tid % G;
  const int units = nr * a.H;
  const size_t row0 = ((size_t)b * a.R + r0) * a.H;  // unit u is row-head row0 + u
  Raw8<T> k[kUnits], v[kUnits];
  auto load = [&](int u0) {
#pragma unroll
    for (int x = 0; x < kUnits; ++x) {
      const int u = min(u0 + x * kGroups + g, units - 1);
      k[x].load(static_cast<const T*>(a.k_rows) + (row0 + u) * DH + gl * 8);
      v[x].load(static_cast<const T*>(a.v_rows) + (row0 + u) * DH + gl * 8);
    }
  };
  load(0);
  if (tid < nr) {
    const int p = pos[r0 + tid];
    if (p < -1 || p >= a.N) set_status(a.status, FDLLM_ERR_BAD_INDEX);
    s_pos[tid] = p >= a.N ? -1 : p;
  }
  __syncthreads();
  if (r0 + 1 < a.R) {  // a later row of the same slot replaces this block's
    int lo = INT_MAX, hi = 0;
    for (int i = 0; i < nr; ++i)
      if (s_pos[i] >= 0) {
        lo = min(lo, s_pos[i]);
        hi = max(hi, s_pos[i]);
      }
    __syncthreads();
    for (int j = r0 + 1 + tid; j < a.R; j += kThreads) {
      const int p = pos[j];
      if (p >= lo && p <= hi)
        for (int i = 0; i < nr && r0 + i < j; ++i)
          if (s_pos[i] == p) s_pos[i] = -1;
    }
    __syncthreads();
  }
  const size_t head0 = (size_t)b * a.H;
  int row = g / a.H, h = g - row * a.H;  // of unit g, then of every kGroups-th
  // whole warps go through the loop together: the shuffles need every lane
  for (int u0 = 0; u0 < units; u0 += kUnits * kGroups) {
    if (u0) load(u0);
#pragma unroll
    for (int x = 0; x < kUnits; ++x) {
      const int p = u0 + x * kGroups + g < units ? s_pos[row] : -1;
      const size_t slot = (head0 + h) * a.N + p;
      for (h += kGroups; h >= a.H; h -= a.H) ++row;
      // the rows' maxima, k in even lanes, v in odd ones: each lane divides for one
      float ka = k[x].top(), va = v[x].top();
      const bool odd = gl & 1;
      float m = fmaxf(odd ? va : ka, __shfl_xor_sync(0xffffffffu, odd ? ka : va, 1));
#pragma unroll
      for (int o = 2; o < G; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = fminf(fmaxf(m, kTiny), FLT_MAX);
      const float inv = __fdiv_rn(kFp8Max, m), scale = __fdiv_rn(m, kFp8Max);
      const float other = __shfl_xor_sync(0xffffffffu, inv, 1);
      float f[8];
      k[x].get(f);
      const uint2 kq = quantise8(f, odd ? other : inv);
      v[x].get(f);
      const uint2 vq = quantise8(f, odd ? inv : other);
      if (p >= 0) {
        *reinterpret_cast<uint2*>(a.k_cache + slot * DH + gl * 8) = kq;
        *reinterpret_cast<uint2*>(a.v_cache + slot * DH + gl * 8) = vq;
        if (gl < 2) (gl ? a.v_scale : a.k_scale)[slot] = scale;
      }
    }
  }
}

// grid B * blocks, as the write; a unit at a time, more CTAs being resident for it
// (measured on 16384 slots read back: two units in flight 88 us, one 76).
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
  const int units = nr * a.H;
  // head after head, rows innermost: neighbouring groups read neighbouring slots
  int h = g / nr, row = g - h * nr;
  for (int u = g; u < units; u += kGroups) {
    const int p = pos[r0 + row], r = row, hd = h;
    for (row += kGroups; row >= nr; row -= nr) ++h;
    if (p < 0 || p >= a.N) {
      if (p != -1) set_status(a.status, FDLLM_ERR_BAD_INDEX);
      continue;
    }
    const size_t slot = (head0 + hd) * a.N + p;
    const uint2 kq = __ldcs(reinterpret_cast<const uint2*>(a.k_cache + slot * DH + gl * 8));
    const uint2 vq = __ldcs(reinterpret_cast<const uint2*>(a.v_cache + slot * DH + gl * 8));
    const float ks = a.k_scale[slot], vs = a.v_scale[slot];
    const size_t dst = (((size_t)b * a.R + r0 + r) * a.H + hd) * DH + gl * 8;
    float f[8];
    dequantise8(kq, ks, f);
    store8(static_cast<T*>(a.k_rows) + dst, f);
    dequantise8(vq, vs, f);
    store8(static_cast<T*>(a.v_rows) + dst, f);
  }
}

// Rows of a CTA's block: two (row, head) pairs to a group (one round of the write, which
// has two in flight; two of the read), and 16 rows where a sequence has so many that the
// scan for replaced rows would otherwise be read too often.
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
