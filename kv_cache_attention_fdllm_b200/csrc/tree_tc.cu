// Attention of a tree of drafted tokens over a cache on the 5th-generation tensor
// cores: a 16-bit cache, or an 8-bit one read as it lies.
//
// Mathematics.  A row is a (node, query head) pair; the g = Hq / Hkv heads of a kv
// head and all nodes share its keys, so an item is (chunk of rows, sequence, kv
// head) and its units are tiles of 128 slots.  With one thread to a slot,
//   S^T [128 slots x NQ rows] = K_tile Q^T,   O^T [dh x NQ] += V_tile^T P^T
// waste nothing on padding when rows are few: the slots are the M of both.  The
// softmax keeps a running maximum per row that is raised only when a tile exceeds
// it by 2^kThresh; l sums the weights in fp32 before they are rounded.  The tree's
// mask is one bit test per score, on the tiles that reach past the sequence.
//
// 8 bits (e4m3 elements, a scale per slot): the elements go to the tensor cores as
// they are, with no conversion pass, because everything else fits around them:
//   - a slot's scale multiplies one row of S^T, i.e. one thread's scores, and for V
//     the weights of that thread;
//   - a bf16 query has 8 significant bits, an e4m3 value 4: q 2^x = q1 + q2 with both
//     e4m3 (x per row, so that its largest is in [128, 256)) is exact down to 2^-10,
//     2^-17 of the row's largest, and S = K q1 + K q2, times 2^-x of the column;
//   - a weight is taken as three e5m2 parts (3 significant bits each, of its fp16
//     value): 9 bits, as bf16 has 8, over a range of 2^31, so that a long flat rest
//     far below a sink keeps its weight.  e4m3 parts would lose it (2^17).  The
//     weights carry the slot's scale, and the running maximum of a row is that of
//     score + log2 of the scale over the slots it sees: its largest product of a weight
//     and a scale uses the range, whatever other rows see, and what is lost of a slot is
//     below 2^-25 of that product.
// The parts are more columns of the same MMAs, and an MMA takes some 80 cycles (its
// 128 x 32 bytes of A) whatever its columns: a tile's 8 take about half of the 1400
// cycles that its bytes take from HBM.  (As separate products they took 20.)
//
// Work split: persistent stream-K.  Units are laid out chunk by chunk, sequence by
// sequence, head by head, tile by tile, from the lengths on the device; CTAs take
// equal contiguous ranges, so any mix of lengths is balanced.  Chunks are outermost:
// CTAs on different chunks of the same slots run at the same time and share them in
// L2.  An item split between CTAs leaves (O, m, l) partials in the workspace; the
// last of its contributors (a counter, nobody waits) merges them in CTA order, so
// results do not depend on timing.
//
//   warp 0      producer: K and V tiles by TMA, with the rows' Q (16 bits) or the slots'
//               scales (8 bits)
//   warp 1      TMEM; lane 0 issues both products
//   warp 2      finisher: counts the partials in; 8 bits: with warp 3 splits the next
//               item's Q into its two e4m3 parts
//   warps 4..   softmax (one group, or two that take turns at the tiles), epilogue, merges
//
// Measured (head size 128, times of calls back to back).  16 bits: 64 sequences of 4096, 32
// heads of 32 nodes, 4.3 GB: 650-713 us, the memory's rate; 8 of up to 2000, 32 heads of 40
// nodes, 239 MB: 61 us, of which 37 are bytes and the rest a CTA's first tile, its two segment
// ends and merges.  8 bits, 8 kv heads of 32 rows: 64 sequences of 1000-4080, 343 MB: 129 us;
// 8 of 16384, 278 MB: 88 us: 2000-2300 cycles a tile, some 10000 more a segment.  (The 8-bit
// instances spill some 50 bytes a thread: 640 threads leave 96 registers each.)
//
// O^T is double-buffered in TMEM (once for each group): an item's result is written
// some tiles into the next item, off the softmax path.
//
// Instructions are the other bound in 8 bits: what a CTA does once a segment (open, close,
// merge, write) runs from cold instruction caches, so rare and once-a-segment code is kept
// out of line and short there.  In 16 bits the same calls cost short items 2 us of 22.
//
// NaN and infinity.  Slots past the sequence's nodes are masked in S and zeroed in V
// (0 x NaN would be NaN).  A node's V that is not finite is zeroed the same way, since
// the tensor cores would spread it to rows that do not see it, and added to the
// outputs of those that do when they are written.
#include <limits.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "tc_common.cuh"
#include "tmap.h"

namespace fdllm {

namespace {

constexpr int kKT = 128;  // slots of a tile
constexpr int kMaxNodes = FDLLM_MAX_TREE_NODES;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -3.0e38f;  // maximum of a row that has seen no slot yet (finite: a
                                   // masked score, -inf, then weighs 2^-inf = 0, not NaN)
constexpr uint32_t kFull = 0xffffffffu;
constexpr size_t kSmemBudget = 227 * 1024;

struct TreeParams {
  int B, N, Hq, Hkv, g, T;
  int n_qc, tn;         // chunks of rows, nodes of a chunk (tn * gs rows)
  int gs, hs;           // query heads of a chunk: g, or with hs = 2 chunks to a node half of them
  int nk, nv;           // stages of the K and V rings
  int keep;             // tiles are read by several chunks
  float qk_scale;       // log2(e) / sqrt(dh)
  const void* q;        // 8-bit cache: read by the splitter
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* cache_len;
  const int32_t* parent;
  const int32_t* n_nodes;
  __nv_bfloat16* out;
  int* status;
  unsigned* cnt;        // [kTreeCounters], zero between calls
  float* partials;      // [grid][2][part_floats]
};

template <int NQ, int DH, bool FP8>
struct Cfg {
  // Softmax threads.  Two groups that take turns at the tiles where a tile's way through
  // one (scores, maximum, weights, each behind a wait) takes longer than its bytes: in 8
  // bits, and in the latency of few rows (measured at 16 rows, one sequence: 22.9 us with
  // one group, 20.0 with two).  Else one group with more registers
  // (32 rows, 64 sequences of 4096: 712 us with two groups, 685 with one).
  static constexpr int kGroups = (FP8 || NQ <= 16) ? 2 : 1;
  static constexpr int kCols = 16;  // rows of a thread
  static constexpr int kGroupThreads = 128 * NQ / kCols;
  static constexpr int kSmx = kGroups * kGroupThreads;
  static constexpr int kFinCols = NQ / (kSmx / 128);  // rows of a thread when results are written
  static constexpr int kFinisher = 2, kFirst = 4;  // warp indices
  static constexpr int kAll = 32 * kFirst + kSmx;
  static constexpr int kNQP = NQ == 48 ? 64 : NQ;  // columns of a TMEM buffer, of P's layout
  static constexpr int kBoxes = FP8 ? 1 : DH / 64;
  static constexpr uint32_t kBoxRow = FP8 ? DH : 128;  // bytes of a slot in a box
  static constexpr uint32_t kBoxBytes = kKT * kBoxRow;
  static constexpr uint32_t kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kQBufs = FP8 ? 2 : 1;
  static constexpr int kQParts = FP8 ? 2 : 1;
  static constexpr uint32_t kQPart = NQ * (FP8 ? DH : DH * 2);
  static constexpr uint32_t kQBytes = (kQBufs * kQParts * kQPart + 1023) / 1024 * 1024;
  // 8 bits: the parts lie side by side as more columns of one product (an MMA takes some
  // 80 cycles, its 128 x 32 bytes of A, whatever its columns): S has 2 NQ, P and O 3 NQ
  static constexpr int kSCols = FP8 ? 2 * NQ : kNQP;
  static constexpr int kOParts = FP8 ? 3 : 1;
  static constexpr int kOCols = FP8 ? 3 * NQ : kNQP;
  static constexpr uint32_t kPRow = FP8 ? 128 : kNQP * 2;  // bytes of a slot in P
  static constexpr uint32_t kPBuf = kKT * kPRow;           // a multiple of 1024
  // A row's largest weight lies at 2^kPOff when its maximum is set, and may grow to 2^kThresh
  // before it is raised (8 bits, the slot's scale with it: below 2^(14 + 1) in fp16 and
  // e5m2).  A larger step would rescale less often but leave less room below
  static constexpr float kThresh = FP8 ? 14.f : 8.f;
  static constexpr float kPOff = FP8 ? 8.f : 0.f;
  static constexpr int kPartFloats = NQ * DH + 2 * NQ + 4;  // O, m, l, flag (and padding)
};

// Shared memory: this block, Q, the P buffers, the K ring, the V ring, the sequences'
// tables, the 8-bit slot scales.  All but the last three are at constant offsets, which
// spares the softmax threads their addresses.
struct Misc {
  static constexpr int kBars = 0;               // 50 mbarriers
  static constexpr int kInts = 400;             // Ints
  static constexpr int kM = 640;                // by group: m_run[64], alpha[64]
  static constexpr int kRed = kM + 2 * 512;     // by group: wred[4][64]
  static constexpr int kSum = kRed + 2 * 1024;  // by group: lred[4][64]
  static constexpr int kSegM = kSum + 2 * 1024; // seg_m, seg_l [2 O buffers][2 groups][64]
  static constexpr int kCol = kSegM + 2 * 1024; // col_off[64]: a row's offset in q and out
  static constexpr int kQsc = kCol + 256;       // 8 bits: qsc[2 Q buffers][32], a row's 2^-x
  static constexpr int kZero = kQsc + 256;      // [64] zeros
  static constexpr int kPar = kZero + 256;      // by group: parents of a sequence's nodes
  static constexpr int kVis = kPar + 2 * kMaxNodes * 4;  // by group: columns that see a node
  static constexpr int kBytes = (kVis + 2 * kMaxNodes * 8 + 1023) / 1024 * 1024;
  // of pre[B + 1], len[B], nn[B]
  __host__ __device__ static constexpr int seq_bytes(int B) { return ((3 * B + 1) * 4 + 15) / 16 * 16; }
};

struct Ints {
  uint32_t tmem;
  int abort;
  int done;           // tiles of the range whose last product is issued
  int merge_u[2];     // first unit of the item in partial slot s that this CTA merges, or -1
  // a closed segment, by O buffer and group: has the group tiles in it, did it meet a node's
  // V that is not finite
  int seg_has[2][2];
  int seg_bad[2][2];
  int bad_run[2];     // the last of the running segment, by group
  // the item of a closed segment, by O buffer and group (every thread of the group writes
  // the same): chunk, sequence, kv head, its first unit, whether the segment is all of it,
  // and the group's last tile in it
  int item[2][2][6];
};
static_assert(sizeof(Ints) <= 240, "Misc::kM");

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// OR of a predicate over `n` threads at named barrier `id`.
__device__ __forceinline__ bool bar_any(int id, int n, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
// 2^x on the special-function unit (flush-to-zero; 2^-inf = 0, NaN stays)
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tmem_ld_chunk(uint32_t taddr, float* v, int w) {
  if (w >= 16)
    tc::tmem_ld16(taddr, v);
  else
    tc::tmem_ld8(taddr, v);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
// two floats as f16 (a in the low half); beyond the largest to infinity
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// e4m3 of two floats (lo in the low byte) and the floats they stand for
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
// one float into shared memory, asynchronously; an arrival on a barrier when all of the
// thread's are there
__device__ __forceinline__ void copy_async4(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
// byte offset `off` of a tile whose rows have `row` bytes (32, 64 or 128), swizzled
__device__ __forceinline__ uint32_t swz(uint32_t off, uint32_t row) {
  return off ^ (((off >> 7) & (row / 16 - 1)) << 4);
}
__device__ __forceinline__ bool not_finite(float x) { return !(fabsf(x) <= 3.4028234663852886e38f); }

// Adds to out[dh row d] of the item's rows [c0, c1) the values of their visible nodes' V
// that are not finite (they were left out of the products).  Kept out of line, like all
// that is rare: code that is not in the instruction cache costs microseconds to fetch.
template <int DH, bool FP8>
__device__ __noinline__ void add_unfit(const TreeParams& p, int qc, int b, int h, int len, int nn,
                                       int c0, int c1, int d) {
  const size_t head = ((size_t)b * p.Hkv + h) * p.N + len;
  const int32_t* parent = p.parent ? p.parent + (size_t)b * p.T : nullptr;
  const int h0 = qc % p.hs * p.gs;  // first of the chunk's heads
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    const int node = qc / p.hs * p.tn + c / p.gs, hd = h0 + c % p.gs;
    if (c >= p.tn * p.gs || node >= nn || hd >= p.g) return;
    float sum = 0.f;
    bool any = false;
#pragma unroll 1
    for (int n = node; n >= 0;) {
      float v;
      if constexpr (FP8)
        v = from_e4m3x2(static_cast<const uint8_t*>(p.v_cache)[(head + n) * DH + d]).x *
            p.v_scale[head + n];
      else
        v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_cache)[(head + n) * DH + d]);
      if (not_finite(v)) {
        sum += v;
        any = true;
      }
      int up = parent ? parent[n] : n - 1;
      if (up < -1 || up >= n) up = -1;
      n = up;
    }
    if (any) {
      __nv_bfloat16* o = p.out + (((size_t)b * p.T + node) * p.Hq + h * p.g + hd) * DH + d;
      *o = __float2bfloat16_rn(__bfloat162float(*o) + sum);
    }
  }
}

// A chunk's Q (bf16; `q`: its first row, the others at col_off, ncol in all) as two e4m3
// parts: q 2^sh = q1 + q2, sh by row so that its largest is in [128, 256): what is lost is
// below 2^-17 of it, whatever the rows beside it hold.  Rows past ncol become zeros.  Warp w
// of W takes every W-th row, up to 16 rows' loads in flight together; `free`: waits until dst
// and unit may be written.  unit takes each row's 2^-sh.
template <int NQ, int DH, int W, typename Free>
__device__ __forceinline__ void split_q(const __nv_bfloat16* q, const int* col_off, int ncol, int w,
                                        uint8_t* dst, float* unit, Free free) {
  constexpr int R = NQ / W;   // rows of a warp
  constexpr int E = DH / 32;  // elements of a lane
  constexpr uint32_t kPart = NQ * DH;
  const int lane = threadIdx.x & 31;
  auto load = [&](int r) {
    uint2 raw = make_uint2(0u, 0u);
    if (r < ncol) {
      const __nv_bfloat16* src = q + col_off[r] + lane * E;
      if constexpr (E == 4)
        raw = *reinterpret_cast<const uint2*>(src);
      else
        raw.x = *reinterpret_cast<const uint32_t*>(src);
    }
    return raw;
  };
  // Two passes, the second of which finds the rows in L1: registers for all of them would
  // unroll the conversions, 11 KB of code that the softmax warps' then has to make room for
  // (64 sequences of 500: 65 us for 71)
  constexpr int M = R < 2 ? R : 2;
  static_assert(R <= 16, "loads in flight");
  // lane x keeps the largest |q| of the warp's row x, as the upper 16 bits of a float:
  // magnitudes compare as whole numbers, what is not finite above all the others
  uint32_t mx = 0u;
  {
    uint2 raw[R];
#pragma unroll
    for (int x = 0; x < R; ++x) raw[x] = load(w + x * W);
#pragma unroll
    for (int x = 0; x < R; ++x) {
      const uint32_t m2 = __vmaxu2(raw[x].x & 0x7fff7fffu, raw[x].y & 0x7fff7fffu);
      const uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
      if (lane == x) mx = m;
    }
  }
  // of rows of zeros and of those that are not finite: 0
  int sh = mx == 0u || mx >= 0x7f80u ? 0 : min(max(7 - ((int)(mx >> 7) - 127), -120), 120);
  free();
  if (lane < R) unit[w + lane * W] = __int_as_float((127 - sh) << 23);
#pragma unroll 1
  for (int x0 = 0; x0 < R; x0 += M) {
    uint2 raw[M];
#pragma unroll
    for (int x = 0; x < M; ++x) raw[x] = load(w + (x0 + x) * W);
#pragma unroll
    for (int x = 0; x < M; ++x) {
      const int r = w + (x0 + x) * W;
      const float up = __int_as_float((127 + __shfl_sync(0xffffffffu, sh, x0 + x)) << 23);
      uint32_t b1 = 0u, b2 = 0u;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const uint32_t q = e < 2 ? raw[x].x : raw[x].y;
        float y0 = __uint_as_float(q << 16) * up, y1 = __uint_as_float(q & 0xffff0000u) * up;
        // what is not finite makes the row NaN (the conversion would saturate it)
        if (not_finite(y0)) y0 = __int_as_float(0x7fffffff);
        if (not_finite(y1)) y1 = __int_as_float(0x7fffffff);
        const uint32_t q1 = e4m3x2(y0, y1);
        const float2 g1 = from_e4m3x2(q1);
        const uint32_t q2 = e4m3x2(y0 - g1.x, y1 - g1.y);
        b1 |= q1 << (8 * e);
        b2 |= q2 << (8 * e);
      }
      const uint32_t off = swz((uint32_t)(r * DH + lane * E), DH);
      if constexpr (E == 4) {
        *reinterpret_cast<uint32_t*>(dst + off) = b1;
        *reinterpret_cast<uint32_t*>(dst + kPart + off) = b2;
      } else {
        *reinterpret_cast<uint16_t*>(dst + off) = (uint16_t)b1;
        *reinterpret_cast<uint16_t*>(dst + kPart + off) = (uint16_t)b2;
      }
    }
  }
}

// A slot's row of V in shared memory (boxes of `row` bytes, `box` bytes apart), behind the
// sequence's nodes (`none`): zeros; of a node: zeros in place of elements that are not
// finite.  Returns whether there were any.
template <bool FP8>
__device__ __forceinline__ bool clean_v_here(uint8_t* at, bool none, int row, int boxes, int box) {
  // an exponent of all ones (an e4m3 of all ones) carries into the sign's place
  constexpr uint32_t ones = FP8 ? 0x7f7f7f7fu : 0x7f807f80u;
  constexpr uint32_t one = FP8 ? 0x01010101u : 0x00800080u;
  constexpr uint32_t sign = FP8 ? 0x80808080u : 0x80008000u;
  uint32_t hit = 0u;
#pragma unroll 1
  for (int x = 0; x < boxes; ++x, at += box)
#pragma unroll 4
    for (int q = 0; q < row; q += 16) {
      uint4* v = reinterpret_cast<uint4*>(at + q);
      if (none) {
        *v = make_uint4(0u, 0u, 0u, 0u);
      } else {
        uint4 w = *v;
        const uint32_t m[4] = {((w.x & ones) + one) & sign, ((w.y & ones) + one) & sign,
                               ((w.z & ones) + one) & sign, ((w.w & ones) + one) & sign};
        if (m[0] | m[1] | m[2] | m[3]) {
          hit = 1u;
          // the sign's place to all of the element's
          constexpr uint32_t width = FP8 ? 0xffu : 0xffffu;
          constexpr int shift = FP8 ? 7 : 15;
          w.x &= ~((m[0] >> shift) * width);
          w.y &= ~((m[1] >> shift) * width);
          w.z &= ~((m[2] >> shift) * width);
          w.w &= ~((m[3] >> shift) * width);
          *v = w;
        }
      }
    }
  return hit != 0u;
}

// Which of a chunk's columns see each node of the sequence: vis[node] bit c, [kMaxNodes][2]
// words, by the n threads of a group; `par` takes the sequence's parents.  A thread a node
// of the chunk adds its columns to itself and its ancestors.
__device__ __forceinline__ void build_seen_here(const TreeParams& p, int node0, int b, int nn,
                                                int t, int n, int bar, int* par,
                                                unsigned long long* vis) {
  tc::named_bar_sync(bar, n);  // nobody reads the old ones any more
  for (int k = t; k < nn; k += n) {
    if (p.parent) par[k] = p.parent[(size_t)b * p.T + k];
    vis[k] = 0ull;
  }
  tc::named_bar_sync(bar, n);
  int node = node0 + t;
  if (t < p.tn && node < nn) {
    const unsigned long long cols = (~0ull >> (64 - p.gs)) << (t * p.gs);
#pragma unroll 1
    while (node >= 0) {
      uint32_t* v = reinterpret_cast<uint32_t*>(vis + node);
      if ((uint32_t)cols) atomicOr(v, (uint32_t)cols);
      if (cols >> 32) atomicOr(v + 1, (uint32_t)(cols >> 32));
      int up = p.parent ? par[node] : node - 1;
      if (up < -1 || up >= node) {
        set_status(p.status, FDLLM_ERR_BAD_INDEX);
        up = -1;
      }
      node = up;
    }
  }
  tc::named_bar_sync(bar, n);
}

// The two out of line in 8 bits (136 us for 141 of 32 rows over 64 sequences of 4096), in
// line in 16 (one row, one sequence of 1024: 22.5 us for 24.4).
template <bool FP8>
__device__ __noinline__ bool clean_v_out(uint8_t* at, bool none, int row, int boxes, int box) {
  return clean_v_here<FP8>(at, none, row, boxes, box);
}
template <bool FP8>
__device__ __forceinline__ bool clean_v(uint8_t* at, bool none, int row, int boxes, int box) {
  if constexpr (FP8)
    return clean_v_out<FP8>(at, none, row, boxes, box);
  else
    return clean_v_here<FP8>(at, none, row, boxes, box);
}
__device__ __noinline__ void build_seen_out(const TreeParams& p, int node0, int b, int nn, int t,
                                            int n, int bar, int* par, unsigned long long* vis) {
  build_seen_here(p, node0, b, nn, t, n, bar, par, vis);
}
template <bool FP8>
__device__ __forceinline__ void build_seen(const TreeParams& p, int node0, int b, int nn, int t,
                                           int n, int bar, int* par, unsigned long long* vis) {
  if constexpr (FP8)
    build_seen_out(p, node0, b, nn, t, n, bar, par, vis);
  else
    build_seen_here(p, node0, b, nn, t, n, bar, par, vis);
}

// tc::mbar_wait with what follows a wait that is not over at once out of line
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return tc::mbar_wait(bar, parity, abort, status);
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         int* status) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  return wait_on(bar, parity, abort, status);
}

// orders this thread's view of memory, device-wide, around an atomic count
__device__ __forceinline__ void fence_gpu() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

// Polling loops give up after kWaitLimitNs without progress.
struct IdleClock {
  uint64_t t0 = 0;
  uint32_t spins = 0;
  __device__ __forceinline__ void reset() { t0 = 0; spins = 0; }
  __device__ __forceinline__ bool idle(volatile int* abort, int* status) {
    if ((++spins & 63u) != 0) return true;
    if (*abort) return false;
    const uint64_t now = global_ns();
    if (t0 == 0) {
      t0 = now;
    } else if (now - t0 > kWaitLimitNs) {
      *abort = 1;
      set_status(status, FDLLM_ERR_TIMEOUT);
      return false;
    }
    return true;
  }
};

// Waits for something that may take a whole item or range: for as long as *done moves, and
// kWaitLimitNs from when it stands still.
__device__ __noinline__ bool wait_while_moving(uint64_t* bar, uint32_t parity, const volatile int* done,
                                               volatile int* abort, int* status) {
  IdleClock clk;
  int seen = *done;
  while (!tc::mbar_try_wait(bar, parity)) {
    const int now = *done;
    if (now != seen) {
      seen = now;
      clk.reset();
    }
    if (!clk.idle(abort, status)) return false;
  }
  return true;
}

// First unit of CTA c's range, and the CTA whose range holds unit u (the largest c
// with lo(c) <= u; a double-precision estimate is put right with exact products).
__device__ __forceinline__ int unit_lo(int total, int G, int c) {
  const long long a = (long long)total * c;
  return a <= INT_MAX ? (int)a / G : (int)(a / G);
}
__device__ __forceinline__ int owner_of(int u, int total, int G) {
  const long long lim = ((long long)u + 1) * G;
  int c = (int)((double)(lim - 1) / (double)total);
  c = c < 0 ? 0 : (c >= G ? G - 1 : c);
  while (c + 1 < G && (long long)total * (c + 1) < lim) ++c;
  while (c > 0 && (long long)total * c >= lim) --c;
  return c;
}

// Where a unit lies: chunk, sequence, kv head, tile; the sequence's tile count.
struct Seqs {
  const int* pre;  // [B + 1] tiles of the sequences in front
  int B, Hkv, total;  // total: tiles of all sequences (pre[B])
};
struct Cursor {
  int qc, b, h, t, tb;
  __device__ __forceinline__ void init(int u, const Seqs& s) {
    const int per = s.total * s.Hkv;
    qc = u / per;
    const int rem = u - qc * per;
    const int tile = rem / s.Hkv;  // b: the last with pre[b] <= tile (its tiles are not 0)
    int lo = 0, hi = s.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s.pre[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    b = lo;
    tb = s.pre[b + 1] - s.pre[b];
    const int r = rem - s.pre[b] * s.Hkv;
    h = r / tb;
    t = r - h * tb;
  }
  __device__ __forceinline__ void next_item(const Seqs& s) {
    t = 0;
    if (++h == s.Hkv) {
      h = 0;
      do {
        if (++b == s.B) {
          b = 0;
          ++qc;
        }
      } while (s.pre[b + 1] == s.pre[b]);
      tb = s.pre[b + 1] - s.pre[b];
    }
  }
  __device__ __forceinline__ void next(const Seqs& s) {
    if (++t == tb) next_item(s);
  }
};

template <int NQ, int DH, bool FP8>
__global__ void __launch_bounds__(Cfg<NQ, DH, FP8>::kAll, 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, TreeParams p) {
  using C = Cfg<NQ, DH, FP8>;
  constexpr int kSmx = C::kSmx;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int NK = p.nk, NV = p.nv;
  uint8_t* misc = smem;
  uint8_t* q_buf = smem + Misc::kBytes;
  uint8_t* p_buf = q_buf + C::kQBytes;
  uint8_t* k_ring = p_buf + 2 * C::kPBuf;
  uint8_t* v_ring = k_ring + NK * C::kTileBytes;
  int* s_pre = reinterpret_cast<int*>(v_ring + NV * C::kTileBytes);
  int* s_len = s_pre + p.B + 1;
  int* s_nn = s_len + p.B;
  // 8 bits, by V stage: the slots' K scales and V scales [2][128]
  float* scales = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(s_pre) + Misc::seq_bytes(p.B));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(misc + Misc::kBars);
  uint64_t* k_empty = k_full + 8;
  uint64_t* v_full = k_empty + 8;
  uint64_t* v_empty = v_full + 8;
  uint64_t* q_full = v_empty + 8;    // [2]
  uint64_t* q_empty = q_full + 2;    // [2]
  uint64_t* s_full = q_empty + 2;    // [2]
  uint64_t* s_empty = s_full + 2;    // [2]
  uint64_t* p_full = s_empty + 2;    // [2]
  uint64_t* pv_done = p_full + 2;    // [2]
  uint64_t* fin_full = pv_done + 2;  // [2] a partial's stores are issued
  uint64_t* seg_full = fin_full + 2; // [2] by O buffer: both groups' O of the segment is final
  uint64_t* o_empty = seg_full + 2;  // [2] by O buffer: its result is written
  Ints* I = reinterpret_cast<Ints*>(misc + Misc::kInts);
  int* abort_flag = &I->abort;
  float* s_mrun = reinterpret_cast<float*>(misc + Misc::kM);
  float* s_wred = reinterpret_cast<float*>(misc + Misc::kRed);
  float* s_lred = reinterpret_cast<float*>(misc + Misc::kSum);
  float* seg_m = reinterpret_cast<float*>(misc + Misc::kSegM);
  float* seg_l = seg_m + 2 * 128;
  int* col_off = reinterpret_cast<int*>(misc + Misc::kCol);
  float* qsc = reinterpret_cast<float*>(misc + Misc::kQsc);  // [2][32]
  float* s_zero = reinterpret_cast<float*>(misc + Misc::kZero);  // [64] zeros
  int* s_par = reinterpret_cast<int*>(misc + Misc::kPar);
  unsigned long long* s_vis = reinterpret_cast<unsigned long long*>(misc + Misc::kVis);

  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  // two S and two O a group
  constexpr uint32_t cols = 2 * C::kSCols + 2 * C::kGroups * C::kOCols;
  constexpr uint32_t ncols = cols <= 128 ? 128 : (cols <= 256 ? 256 : 512);
  static_assert(cols <= 512, "TMEM");

  if (tid == 0) {
    for (int s = 0; s < 8; ++s) {
      tc::mbar_init(&k_full[s], 1);
      tc::mbar_init(&k_empty[s], 1);
      tc::mbar_init(&v_full[s], FP8 ? 33 : 1);  // 8 bits: every lane's scales
      tc::mbar_init(&v_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&q_full[b], FP8 ? 2 : 1);  // 8 bits: the two warps that split Q
      tc::mbar_init(&q_empty[b], 1 + (FP8 ? kSmx / 32 : 0));  // 8 bits: the scales' readers too
      tc::mbar_init(&s_full[b], 1);
      tc::mbar_init(&s_empty[b], C::kGroupThreads / 32);
      tc::mbar_init(&p_full[b], C::kGroupThreads / 32);
      tc::mbar_init(&seg_full[b], kSmx / 32);
      tc::mbar_init(&o_empty[b], kSmx / 32);
      tc::mbar_init(&pv_done[b], 1);
      tc::mbar_init(&fin_full[b], kSmx / 32);
    }
    I->abort = 0;
    I->done = 0;
    I->bad_run[0] = I->bad_run[1] = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(&I->tmem, ncols);
  if (tid < 64) {
    s_zero[tid] = 0.f;
    const int n = tid / p.gs;
    col_off[tid] = (n * p.Hq + tid - n * p.gs) * DH;
  }
  // rows of Q past the chunk's: zeros, whatever the product makes of them is not read
  for (int i = tid; i < (int)(C::kQBytes / 16); i += C::kAll)
    reinterpret_cast<uint4*>(q_buf)[i] = make_uint4(0u, 0u, 0u, 0u);
  tc::fence_proxy_async_smem();
  if (tid == 64) {
    tc::prefetch_tmap(&tm_k);
    tc::prefetch_tmap(&tm_v);
    if (!FP8) tc::prefetch_tmap(&tm_q);
  }
  // nothing that an earlier kernel wrote is read before this
  tc::griddep_wait();
  for (int b = tid; b < p.B; b += C::kAll) {
    int len = p.cache_len[b];
    int nn = p.n_nodes ? p.n_nodes[b] : p.T;
    if (len < 0 || nn < 0 || nn > p.T || len > p.N - nn) {
      if (cta == 0) set_status(p.status, FDLLM_ERR_BAD_INDEX);
      len = 0;
      nn = 0;
    }
    s_len[b] = len;
    s_nn[b] = nn;
  }
  __syncthreads();
  if (warp == 0) {
    int run = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      int x = b < p.B && s_nn[b] > 0 ? (s_len[b] + s_nn[b] + kKT - 1) / kKT : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < p.B) s_pre[b + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) s_pre[0] = 0;
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = I->tmem;
  const uint32_t tmem_o = tmem + 2 * C::kSCols;
  Seqs S;
  S.pre = s_pre;
  S.B = p.B;
  S.Hkv = p.Hkv;
  S.total = s_pre[p.B];
  const int U = S.total * p.Hkv * p.n_qc;  // fits: checked on the host for the largest
  const int G = min((int)gridDim.x, U);
  const int u0 = cta < G ? unit_lo(U, G, cta) : 0;
  const int u1 = cta < G ? unit_lo(U, G, cta + 1) : 0;
  const int T = u1 - u0;

  // Where a chunk's first row is in q and out, and how many columns are rows of the sequence
  // (with hs = 2 a chunk has one node).
  auto row_of = [&](int qc, int b, int h) {
    return (((size_t)b * p.T + qc / p.hs * p.tn) * p.Hq + h * p.g + qc % p.hs * p.gs) * DH;
  };
  auto columns = [&](int qc, int b) {
    return min(p.tn, s_nn[b] - qc / p.hs * p.tn) * min(p.gs, p.g - qc % p.hs * p.gs);
  };

  if (T == 0) {
    // no work for this CTA (it meets the others at the end)
  } else if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    // K and V each have their own ring, filled as soon as a stage frees; 16 bits: the one
    // Q buffer takes the next item's rows as soon as the last QK of the running one is
    // done.  8 bits: the slots' scales come with the V tiles, 4-byte copies by every lane
    // (a head's scales start anywhere).
    {
      const bool leader = lane == 0;
      const uint64_t pol_kv = p.keep ? tc::policy_evict_normal() : tc::policy_evict_first();
      const uint64_t pol_q = tc::policy_evict_last();
      int ik = 0, iv = 0, qn = 0, ks = 0, vs = 0;
      uint32_t kph = 1u, vph = 1u;
      Cursor ck, cv, cq;
      ck.init(u0, S);
      cv = ck;
      cq = ck;
      int q_left = FP8 ? 0 : T;  // units not yet covered by a loaded Q
      IdleClock clk;
      while (iv < T || q_left > 0) {
        bool progressed = false;
        if constexpr (!FP8) {
          if (q_left > 0 && __all_sync(kFull, tc::mbar_test(&q_empty[0], ((uint32_t)qn & 1u) ^ 1u))) {
            if (leader) {
              const uint32_t bytes = (uint32_t)(p.tn * p.g) * 128u;
              tc::mbar_arrive_expect_tx(&q_full[0], bytes * C::kBoxes);
#pragma unroll
              for (int x = 0; x < C::kBoxes; ++x)
                tc::tma_load_5d(q_buf + x * NQ * 128, &tm_q, &q_full[0], x * 64, 0, cq.h,
                                cq.qc * p.tn, cq.b, pol_q);
            }
            q_left -= cq.tb - cq.t;
            if (q_left > 0) cq.next_item(S);
            ++qn;
            progressed = true;
          }
        }
        if (ik < T && __all_sync(kFull, tc::mbar_test(&k_empty[ks], kph))) {
          if (leader) {
            uint8_t* kd = k_ring + ks * C::kTileBytes;
            tc::mbar_arrive_expect_tx(&k_full[ks], C::kTileBytes);
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x)
              tc::tma_load_3d(kd + x * C::kBoxBytes, &tm_k, &k_full[ks], x * 64, ck.t * kKT,
                              ck.b * p.Hkv + ck.h, pol_kv);
          }
          if (++ks == NK) {
            ks = 0;
            kph ^= 1u;
          }
          if (++ik < T) ck.next(S);
          progressed = true;
        }
        if (iv < ik && __all_sync(kFull, tc::mbar_test(&v_empty[vs], vph))) {
          if (leader) {
            uint8_t* vd = v_ring + vs * C::kTileBytes;
            tc::mbar_arrive_expect_tx(&v_full[vs], C::kTileBytes);
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x)
              tc::tma_load_3d(vd + x * C::kBoxBytes, &tm_v, &v_full[vs], x * 64, cv.t * kKT,
                              cv.b * p.Hkv + cv.h, pol_kv);
          }
          if constexpr (FP8) {
            const size_t head = ((size_t)cv.b * p.Hkv + cv.h) * p.N;
            float* dst = scales + vs * 256;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int slot = x * 32 + lane;
              const size_t at = head + min(cv.t * kKT + slot, p.N - 1);
              copy_async4(dst + slot, p.k_scale + at);
              copy_async4(dst + 128 + slot, p.v_scale + at);
            }
            copy_async_arrive(&v_full[vs]);
          }
          if (++vs == NV) {
            vs = 0;
            vph ^= 1u;
          }
          if (++iv < T) cv.next(S);
          progressed = true;
        }
        if (!progressed && __any_sync(kFull, !clk.idle(abort_flag, p.status))) break;
        if (progressed) clk.reset();
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // Two in-order streams, QK(i) and PV(j), each issued as soon as its inputs are
    // ready.  The whole warp runs this, converged, and lane 0 alone issues: descriptors
    // then stay in uniform registers, where the instruction wants them.  (Issued from a
    // lane's own branch an MMA cost 77 cycles, more than the tensor cores take for it.)
    constexpr uint32_t swz_code = C::kBoxRow == 128 ? 2u : 4u;
    constexpr uint32_t p_swz = C::kPRow == 128 ? 2u : (C::kPRow == 64 ? 4u : 6u);
    constexpr uint32_t full = kFull;
    const bool leader = lane == 0;
    const uint32_t k_base = tc::smem_u32(k_ring), v_base = tc::smem_u32(v_ring);
    const uint32_t q_base = tc::smem_u32(q_buf), p_base = tc::smem_u32(p_buf);
    const uint32_t t_s = __shfl_sync(full, tmem, 0), t_o = t_s + 2 * C::kSCols;
    int iq = 0, ip = 0, seg = -1, pseg = -1;
    int ks = 0, vs = 0;           // stages of QK(iq) and PV(ip),
    uint32_t kph = 0, vph = 0;    // and their phases
    int seg_i0 = 0;               // range index of segment pseg's first tile
    Cursor cq, cpv;
    cq.init(u0, S);
    cpv = cq;
    // tiles left of the item that QK, PV is in
    int q_left = __shfl_sync(full, min(cq.tb - cq.t, T), 0), pv_left = q_left;
    bool q_opens = true, pv_opens = true;
    IdleClock clk;
    while (ip < T) {
      bool progressed = false;
      if (iq < T) {
        const int qseg = q_opens ? seg + 1 : seg;
        const int qb = C::kQBufs == 2 ? qseg & 1 : 0;
        const int sb = iq & 1;
        const bool ready = tc::mbar_test(&k_full[ks], kph) &&
                           tc::mbar_test(&s_empty[sb], ((uint32_t)(iq >> 1) & 1u) ^ 1u) &&
                           (!q_opens || tc::mbar_test(&q_full[qb], (uint32_t)(qseg / C::kQBufs) & 1u));
        if (__all_sync(full, ready)) {
          seg = qseg;
          tc::tc_fence_after();
          const uint32_t k_addr = k_base + ks * C::kTileBytes;
          const uint32_t q_addr = q_base + qb * (C::kQParts * C::kQPart);
          const uint32_t d = t_s + sb * C::kSCols;
          if constexpr (FP8) {
            constexpr uint32_t idesc = tc::idesc_f8(kKT, C::kSCols, false);
            const uint64_t dk = tc::smem_desc(k_addr, 16, 8 * DH, swz_code);
            const uint64_t dq = tc::smem_desc(q_addr, 16, 8 * DH, swz_code);
#pragma unroll
            for (int kk = 0; kk < DH / 32; ++kk)
              if (leader) tc::mma_f8(d, dk + kk * 2, dq + kk * 2, idesc, kk != 0);
          } else {
            constexpr uint32_t idesc = tc::idesc_bf16(kKT, NQ, false, false);
            const uint64_t dk = tc::smem_desc(k_addr, 16, 1024, 2);
            const uint64_t dq = tc::smem_desc(q_addr, 16, 1024, 2);
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk)
              if (leader)
                tc::mma_bf16(d, dk + ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) / 16,
                             dq + ((kk >> 2) * NQ * 128 + (kk & 3) * 32) / 16, idesc, kk != 0);
          }
          const bool closes = --q_left == 0;
          if (leader) {
            tc::mma_commit(&s_full[sb]);
            tc::mma_commit(&k_empty[ks]);
            if (closes) tc::mma_commit(&q_empty[qb]);
          }
          if (++ks == NK) {
            ks = 0;
            kph ^= 1u;
          }
          ++iq;
          q_opens = closes;
          if (closes && iq < T) {
            cq.next_item(S);
            q_left = __shfl_sync(full, min(cq.tb, T - iq), 0);
          }
          progressed = true;
        }
      }
      if (ip < iq) {
        const bool ready =
            tc::mbar_test(&p_full[ip & 1], (uint32_t)(ip >> 1) & 1u) &&
            tc::mbar_test(&v_full[vs], vph) &&
            (!pv_opens || tc::mbar_test(&o_empty[(pseg + 1) & 1], ((uint32_t)((pseg + 1) >> 1) & 1u) ^ 1u));
        if (__all_sync(full, ready)) {
          if (pv_opens) {
            ++pseg;
            seg_i0 = ip;
          }
          const uint32_t set = ip - seg_i0 < C::kGroups;  // the group's first tile: O is set
          tc::tc_fence_after();
          const uint32_t v_addr = v_base + vs * C::kTileBytes;
          const uint32_t pb_addr = p_base + (ip & 1) * C::kPBuf;
          const uint32_t o_addr =
              t_o + (uint32_t)(((pseg & 1) * C::kGroups + (C::kGroups == 2 ? ip & 1 : 0)) * C::kOCols);
          if constexpr (FP8) {
            constexpr uint32_t idesc = tc::idesc_f8(kKT, C::kOCols, true, true, true);
            const uint64_t dv = tc::smem_desc(v_addr, 0, 8 * DH, swz_code);
            const uint64_t dp = tc::smem_desc(pb_addr, 0, 8 * C::kPRow, p_swz);
#pragma unroll
            for (int kk = 0; kk < kKT / 32; ++kk)
              if (leader)
                tc::mma_f8(o_addr, dv + kk * 2 * DH, dp + kk * 2 * C::kPRow, idesc,
                           kk == 0 ? set ^ 1u : 1u);
          } else {
            constexpr uint32_t idesc = tc::idesc_bf16(kKT, NQ, true, true);
            const uint64_t dv = tc::smem_desc(v_addr, DH == 128 ? 16384 : 0, 1024, 2);
            const uint64_t dp = tc::smem_desc(pb_addr, 0, 8 * C::kPRow, p_swz);
#pragma unroll
            for (int kk = 0; kk < kKT / 16; ++kk)
              if (leader)
                tc::mma_bf16(o_addr, dv + kk * 128, dp + kk * C::kPRow, idesc,
                             kk == 0 ? set ^ 1u : 1u);
          }
          const bool closes = --pv_left == 0;
          if (leader) {
            tc::mma_commit(&pv_done[ip & 1]);
            tc::mma_commit(&v_empty[vs]);
            *reinterpret_cast<volatile int*>(&I->done) = ip + 1;
          }
          if (++vs == NV) {
            vs = 0;
            vph ^= 1u;
          }
          ++ip;
          pv_opens = closes;
          if (closes && ip < T) {
            cpv.next_item(S);
            pv_left = __shfl_sync(full, min(cpv.tb, T - ip), 0);
          }
          progressed = true;
        }
      }
      if (!progressed && __any_sync(full, !clk.idle(abort_flag, p.status))) break;
      if (progressed) clk.reset();
    }
  } else if (warp >= C::kFirst) {
    // ------------------------------------------------------------ softmax / epilogue
    // Group `grp` takes the tiles with its parity (all of them when there is one
    // group).  Its warps that share a TMEM lane quarter split the rows: a thread owns
    // one slot and the columns [c0, c0 + 16); when results are written, one dh row and
    // the columns [f0, f0 + NF).
    constexpr int NQH = C::kCols, NF = C::kFinCols, GT = C::kGroupThreads, KG = C::kGroups;
    const int st = tid - 32 * C::kFirst;     // 0..kSmx-1
    const int grp = KG == 2 ? st / GT : 0;
    const int gt = st - grp * GT;
    const int quarter = warp & 3;
    const int c0 = (gt >> 7) * NQH;
    const int f0 = (st >> 7) * NF;
    const int kl = quarter * 32 + lane;      // TMEM lane: slot of S^T, dh row of O^T
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const int bar_a = 1 + 2 * grp, bar_b = 2 + 2 * grp;  // named barriers of the group
    constexpr int kBarCount = 5, kBarAll = 6;
    float* m_run = s_mrun + grp * 128;  // [64], then the rescales of l and O
    float* alpha = m_run + 64;
    float* wred = s_wred + grp * 256;  // [4][64]
    // a segment's sums of l by warp.  Not in wred's place: the next segment's first tile
    // writes there without a barrier behind the reads of these
    float* lred = s_lred + grp * 256;
    unsigned long long* vis = s_vis + grp * kMaxNodes;
    int* par = s_par + grp * kMaxNodes;
    float l[NQH];
    int vis_key = -1;      // (chunk, sequence) that vis stands for
    int pv_waited = -1;    // index of the last PV this thread waited for
    Cursor cs;
    cs.init(u0, S);
    const int item0 = u0 - cs.t;  // first unit of the item the range starts in

    auto wait_pv = [&](int e) {
      if (e >= 0 && pv_waited < e) {
        // after a timeout every later wait returns at once: keep going, so that all
        // threads still meet at the same barriers
        wait_bar(&pv_done[e & 1], (uint32_t)(e >> 1) & 1u, abort_flag, p.status);
        pv_waited = e;
      }
    };

    // The last segment this group closed, and what has become of it.
    int d_seg = -1;
    bool d_pub = true, d_fin = true;

    // Tells the other group that this one's O of the closed segment is final.
    auto publish = [&]() {
      wait_pv(I->item[d_seg & 1][grp][5]);
      tc::tc_fence_after();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&seg_full[d_seg & 1]);
      d_pub = true;
    };
    // Writes the closed segment's result from both groups' O: the output of a whole
    // item, or this CTA's partial of a split one, whose arrival on fin_full hands it to
    // the finisher.
    auto finish = [&]() {
      const int sl = d_seg & 1;
      const int* it = I->item[sl][grp];
      const int d_qc = it[0], d_b = it[1], d_h = it[2];
      wait_bar(&seg_full[sl], (uint32_t)(d_seg >> 1) & 1u, abort_flag, p.status);
      tc::tc_fence_after();
      const float* sm = seg_m + sl * 128;  // [group][64]
      const float* ls = seg_l + sl * 128;
      float o[NF];
      bool bad = false;
#pragma unroll
      for (int x = 0; x < KG; ++x) {
        // a group without a tile in the segment has left its O as it was
        const bool has = I->seg_has[sl][x] != 0;
        bad |= I->seg_bad[sl][x] != 0;
        float y[NF], z[C::kOParts > 1 ? 2 * NF : 1];
        const uint32_t at = tmem_o + (uint32_t)((sl * KG + x) * C::kOCols) + lane_off + (uint32_t)f0;
        tmem_ld_chunk(at, y, NF);
        if constexpr (C::kOParts > 1) {
          tmem_ld_chunk(at + NQ, z, NF);
          tmem_ld_chunk(at + 2 * NQ, z + NF, NF);
        }
        tc::tmem_wait_ld();
        if constexpr (C::kOParts > 1) {
#pragma unroll
          for (int c = 0; c < NF; ++c) y[c] += z[c] + z[NF + c];
        }
#pragma unroll
        for (int c = 0; c < NF; ++c) {
          float w = 1.f;
          if (KG == 2) w = ex2_approx(sm[x * 64 + f0 + c] - fmaxf(sm[f0 + c], sm[64 + f0 + c]));
          const float v = has ? y[c] * w : 0.f;
          o[c] = x == 0 ? v : o[c] + v;
        }
      }
      auto sums = [&](int c) {  // l of column c, both groups at the larger maximum
        if (KG == 1) return ls[c];
        const float M = fmaxf(sm[c], sm[64 + c]);
        return ex2_approx(sm[c] - M) * ls[c] + ex2_approx(sm[64 + c] - M) * ls[64 + c];
      };
      if (it[4]) {
        __nv_bfloat16* o_at = p.out + row_of(d_qc, d_b, d_h) + kl;
        const int ncol = columns(d_qc, d_b);
        if (kl < DH) {
#pragma unroll
          for (int c = 0; c < NF; ++c)
            if (f0 + c < ncol)
              o_at[col_off[f0 + c]] = __float2bfloat16_rn(__fdividef(o[c], sums(f0 + c)));
          if (bad) add_unfit<DH, FP8>(p, d_qc, d_b, d_h, s_len[d_b], s_nn[d_b], f0, f0 + NF, kl);
        }
      } else {
        // slot 0 for the item the range starts in, 1 for the one it ends in
        const int slot = (it[3] == item0) ? 0 : 1;
        float* part = p.partials + ((size_t)cta * 2 + slot) * C::kPartFloats;
        if (kl < DH) {
          // O as [NQ / 4][dh row][4]: a warp's 16-byte accesses are consecutive
          float4* dst = reinterpret_cast<float4*>(part) + f0 / 4 * DH + kl;
#pragma unroll
          for (int v = 0; v < NF / 4; ++v)
            dst[v * DH] = make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
        }
        if (st < NQ) {
          part[(size_t)NQ * DH + st] = KG == 1 ? sm[st] : fmaxf(sm[st], sm[64 + st]);
          part[(size_t)NQ * DH + NQ + st] = sums(st);
        }
        if (st == 0) part[(size_t)NQ * DH + 2 * NQ] = bad ? 1.f : 0.f;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&fin_full[slot]);
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&o_empty[sl]);
      d_fin = true;
    };

    int i0 = 0;  // range index of the segment's first tile
    int vst = grp;  // V stage of the group's next tile, and its phase
    uint32_t vph = 0u;
    if constexpr (FP8) {
      // the range's first Q is split by all of these warps: nothing else is to do yet
      split_q<NQ, DH, C::kSmx / 32>(
          static_cast<const __nv_bfloat16*>(p.q) + row_of(cs.qc, cs.b, cs.h), col_off,
          columns(cs.qc, cs.b), warp - C::kFirst, q_buf, qsc, [] {});
      tc::fence_proxy_async_smem();
      tc::named_bar_sync(kBarAll, C::kSmx);
      if (st < 64 && lane == 0) tc::mbar_arrive(&q_full[0]);  // twice
    }

    for (int seg = 0;; ++seg) {
      // ---- a segment: the tiles [i0, i0 + nt) of one item; behind the last an empty one
      const int nt = min(cs.tb - cs.t, T - i0);
      const int qc = cs.qc, b = cs.b;
      const int len = s_len[b], lim = len + s_nn[b];
      bool first = true;
      int last = -1;
#pragma unroll
      for (int c = 0; c < NQH; ++c) l[c] = 0.f;
#pragma unroll 1
      for (int i = KG == 2 ? i0 + ((i0 ^ grp) & 1) : i0;; i += KG) {
        const bool closing = i + KG >= i0 + nt;
        if (i < i0 + nt) {
          const int t = cs.t + i - i0;
          const bool tree = (t + 1) * kKT > len;  // the tile holds nodes (or slots past them)
          if (tree && b * p.n_qc + qc != vis_key) {
            vis_key = b * p.n_qc + qc;
            build_seen<FP8>(p, qc / p.hs * p.tn, b, s_nn[b], gt, GT, bar_a, par, vis);
          }
          const int slot = t * kKT + kl;
          const bool zero_v = tree && slot >= lim;  // this slot's V goes into no sum
          uint32_t seen = ~0u;                      // columns that see the slot
          if (tree && slot >= len)
            seen = slot < lim ? (uint32_t)(vis[slot - len] >> c0) : 0u;

          const int sb = i & 1;
          wait_bar(&s_full[sb], (uint32_t)(i >> 1) & 1u, abort_flag, p.status);
          tc::tc_fence_after();
          float ksc = p.qk_scale, vs = 1.f, vexp = 0.f;
          if constexpr (FP8) {
            wait_bar(&v_full[vst], vph, abort_flag, p.status);
            const float* sc = scales + vst * 256 + kl;
            ksc *= sc[0];
            vs = sc[128];
            // exponent of the slot's V scale: 2^vexp <= |vs| < 2^(vexp + 1).  At least 2^-84,
            // for zeros too (rows all of smaller ones lose bits below 2^-33 of that; l stays
            // below 2^(14 + 84) a slot); a scale that is not finite weighs nothing here
            const int eb = (__float_as_int(vs) >> 23) & 255;
            vexp = (float)(eb < 255 ? max(eb - 127, -84) : -84);
          }

          // ---- scores (log2 units) against the running maximum: row kl of S^T, this
          // thread's columns.  The maximum is raised when a weight (8 bits: times the slot's
          // scale) exceeds 2^kThresh (masked ones never do); a segment's first tile sets it.  For that the
          // scores are formed again as they are (pass 1): one copy of the code, S being there
          // until the end.
          float d[NQH];  // exponents of the weights
          int pass = first ? 1 : 0;
          bool any = first;
#pragma unroll 1
          for (;;) {
            const uint32_t at = tmem + lane_off + sb * C::kSCols + c0;
#pragma unroll
            for (int c = 0; c < NQH; c += 16) tmem_ld_chunk(at + c, d + c, 16);
            if constexpr (FP8) {
              float d2[NQH];
#pragma unroll
              for (int c = 0; c < NQH; c += 16) tmem_ld_chunk(at + NQ + c, d2 + c, 16);
              tc::tmem_wait_ld();
              const float4* u4 = reinterpret_cast<const float4*>(qsc + (seg & 1) * 32 + c0);
#pragma unroll
              for (int c = 0; c < NQH; c += 4) {
                const float4 u = u4[c / 4];
                d[c] = (d[c] + d2[c]) * u.x;
                d[c + 1] = (d[c + 1] + d2[c + 1]) * u.y;
                d[c + 2] = (d[c + 2] + d2[c + 2]) * u.z;
                d[c + 3] = (d[c + 3] + d2[c + 3]) * u.w;
              }
            } else {
              tc::tmem_wait_ld();
            }
            const float4* m4 = reinterpret_cast<const float4*>((pass == 1 ? s_zero : m_run) + c0);
#pragma unroll
            for (int c = 0; c < NQH; c += 4) {
              const float4 m = m4[c / 4];
              d[c] = fmaf(d[c], ksc, -m.x);
              d[c + 1] = fmaf(d[c + 1], ksc, -m.y);
              d[c + 2] = fmaf(d[c + 2], ksc, -m.z);
              d[c + 3] = fmaf(d[c + 3], ksc, -m.w);
            }
            if (tree) {
#pragma unroll
              for (int c = 0; c < NQH; ++c)
                if (!((seen >> c) & 1u)) d[c] = -INFINITY;
            }
            if (pass == 0) {
              float top = d[0];
#pragma unroll
              for (int c = 1; c < NQH; ++c) top = fmaxf(top, d[c]);
              if (FP8) top += vexp;
              any = bar_any(bar_b, GT, top > C::kThresh);
              if (!any) break;
              pass = 1;
              continue;
            }
#pragma unroll
            for (int c = 0; c < NQH; ++c) {
              const float wm = warp_max(FP8 ? d[c] + vexp : d[c]);
              if (lane == c) wred[quarter * 64 + c0 + c] = wm;
            }
            tc::named_bar_sync(bar_a, GT);
            if (gt < NQ) {
              const float mo = first ? kNone : m_run[gt];
              const float tm = fmaxf(fmaxf(wred[gt], wred[64 + gt]), fmaxf(wred[128 + gt], wred[192 + gt]));
              const float mn = (tm - mo > C::kThresh) ? tm - C::kPOff : mo;
              alpha[gt] = ex2_approx(mo - mn);
              m_run[gt] = mn;
            }
            tc::named_bar_sync(bar_a, GT);
#pragma unroll
            for (int c = 0; c < NQH; ++c) {
              l[c] *= alpha[c0 + c];
              d[c] -= m_run[c0 + c];
            }
            break;
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&s_empty[sb]);

          // ---- P buffer i&1 is free once PV(i-2) is done; rescaling O needs the group's
          // last PV
          wait_pv(i - 2);
          if (any && !first) {
            if (KG == 1) wait_pv(i - 1);
            tc::tc_fence_after();
            const uint32_t at =
                tmem_o + (uint32_t)(((seg & 1) * KG + grp) * C::kOCols) + lane_off + (uint32_t)c0;
            float o[8];
#pragma unroll 1
            for (int cc = 0; cc < C::kOParts * NQH; cc += 8) {
              const int c1 = cc & (NQH - 1), part = cc / NQH;
              tc::tmem_ld8(at + part * NQ + c1, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 8; ++c) o[c] *= alpha[c0 + c1 + c];
              tc::tmem_st8(at + part * NQ + c1, o);
            }
            tc::tmem_wait_st();
          }
          if (tree && slot >= len && c0 == 0) {
            // V of a slot past the nodes: zeros; of a node: zeros in place of what is not
            // finite
            wait_bar(&v_full[vst], vph, abort_flag, p.status);
            if (clean_v<FP8>(v_ring + vst * C::kTileBytes + kl * C::kBoxRow, zero_v, C::kBoxRow,
                             C::kBoxes, C::kBoxBytes) ||
                (FP8 && !zero_v && not_finite(vs)))
              I->bad_run[grp] = 1;
          }

          // ---- P = 2^(s - m) into row kl of the MN-major swizzled P^T tile
          uint8_t* pb = p_buf + (i & 1) * C::kPBuf;
          if constexpr (FP8) {
            // the weight carries the slot's scale
            const float w = zero_v || (tree && slot >= len && not_finite(vs)) ? 0.f : vs;
            uint32_t pk[3][NQH / 4];
#pragma unroll
            for (int c = 0; c < NQH; c += 4) {
              uint32_t hp[2][3];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float p0 = ex2_approx(d[c + 2 * y]);
                const float p1 = ex2_approx(d[c + 2 * y + 1]);
                l[c + 2 * y] += p0;
                l[c + 2 * y + 1] += p1;
                // fp16 value h; its upper byte is e5m2, cut off: h = hi + rest, twice; the
                // last part is rounded (half a unit added below the byte; it never carries
                // past 16 bits, parts being far below the largest)
                const uint32_t h = pack_f16x2(p0 * w, p1 * w);
                const uint32_t h1 = h & 0xff00ff00u;
                const uint32_t r1 = sub_f16x2(h, h1);
                const uint32_t h2 = r1 & 0xff00ff00u;
                const uint32_t r2 = sub_f16x2(r1, h2);
                hp[y][0] = h1;
                hp[y][1] = h2;
                hp[y][2] = r2 + 0x00800080u;
              }
#pragma unroll
              for (int part = 0; part < 3; ++part)
                pk[part][c / 4] = __byte_perm(hp[0][part], hp[1][part], 0x7531);
            }
#pragma unroll
            for (int part = 0; part < 3; ++part)
#pragma unroll
              for (int ch = 0; ch < NQH / 16; ++ch)
                *reinterpret_cast<uint4*>(
                    pb + swz((uint32_t)(kl * C::kPRow + part * NQ + c0 + ch * 16), C::kPRow)) =
                    make_uint4(pk[part][4 * ch], pk[part][4 * ch + 1], pk[part][4 * ch + 2],
                               pk[part][4 * ch + 3]);
          } else {
            uint32_t pk[NQH / 2];
#pragma unroll
            for (int c = 0; c < NQH; c += 2) {
              const float p0 = ex2_approx(d[c]);
              const float p1 = ex2_approx(d[c + 1]);
              l[c] += p0;
              l[c + 1] += p1;
              pk[c / 2] = pack_bf16x2(p0, p1);
            }
#pragma unroll
            for (int ch = 0; ch < NQH / 8; ++ch)
              *reinterpret_cast<uint4*>(pb + swz((uint32_t)(kl * C::kPRow + c0 * 2 + ch * 16), C::kPRow)) =
                  make_uint4(pk[ch * 4], pk[ch * 4 + 1], pk[ch * 4 + 2], pk[ch * 4 + 3]);
          }
          tc::fence_proxy_async_smem();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&p_full[i & 1]);
          first = false;
          last = i;
          vst += KG;
          if (vst >= NV) {
            vst -= NV;
            vph ^= 1u;
          }
        }

        // ---- the segment before: final once its last PV is two tiles back, written a
        // tile later, off this one's path; at the latest when this one is closed, whose
        // successor reuses its O
        do {
          if (!d_pub)
            publish();
          else if (!d_fin)
            finish();
        } while (closing && !d_fin);
        if (closing) break;
      }
      if (i0 == T) break;

      // ---- close the segment
      if (last >= 0) {
        // l summed over the warp's slots: each round gives half of the columns away, so that
        // a pair of lanes ends with one column's sum
        static_assert(NQH == 16, "16 columns a thread");
#pragma unroll
        for (int o = 16, w = 8; w >= 1; o >>= 1, w >>= 1) {
          const bool up = lane & o;
#pragma unroll
          for (int c = 0; c < w; ++c) {
            const float mine = up ? l[c + w] : l[c], gone = up ? l[c] : l[c + w];
            l[c] = mine + __shfl_xor_sync(0xffffffffu, gone, o);
          }
        }
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], 1);
        if (!(lane & 1)) lred[quarter * 64 + c0 + (lane >> 1)] = l[0];
        tc::named_bar_sync(bar_a, GT);
      }
      const int sl = seg & 1;
      if (gt < NQ) {
        seg_m[sl * 128 + grp * 64 + gt] = last >= 0 ? m_run[gt] : kNone;
        seg_l[sl * 128 + grp * 64 + gt] =
            last >= 0 ? lred[gt] + lred[64 + gt] + lred[128 + gt] + lred[192 + gt] : 0.f;
      }
      if (gt == 0) {
        I->seg_has[sl][grp] = last >= 0;
        I->seg_bad[sl][grp] = I->bad_run[grp];
        I->bad_run[grp] = 0;
      }
      if constexpr (FP8) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&q_empty[seg & 1]);  // the scales of Q are read
      }
      d_seg = seg;
      int* it = I->item[sl][grp];
      it[0] = qc;
      it[1] = b;
      it[2] = cs.h;
      it[3] = u0 + i0 - cs.t;
      it[4] = cs.t == 0 && nt == cs.tb;
      it[5] = last;
      d_pub = d_fin = false;
      i0 += nt;
      if (i0 < T) {
        cs.next_item(S);
      }
    }

    // ---- the finisher has taken the counts of this CTA's partials
    tc::named_bar_sync(kBarCount, C::kSmx + 32);
#pragma unroll 1
    for (int slot = 0; slot < 2; ++slot) {
      const int iu = I->merge_u[slot];
      if (iu < 0) continue;
      // ---- merge an item whose contributors have all stored their partials, in CTA
      // order: with M the largest m_j, O = sum 2^(m_j - M) O_j / sum 2^(m_j - M) l_j.  A
      // thread takes 8 columns of its dh row at a time and folds the contributors in
      // rounds whose loads are all issued before the first is used: one round trip to L2
      // a round, and no barrier.  (Read around L1: the finisher's fence and the barrier
      // above order these loads behind the stores.)
      Cursor at;
      at.init(iu, S);
      const int c_first = owner_of(iu, U, G), c_last = owner_of(iu + at.tb - 1, U, G);
      const int n_c = c_last - c_first + 1;
      // the item is slot 0 of a contributor whose range starts inside it
      const long long iu_g = (long long)iu * G;
      auto part_of = [&](int j) -> const float* {
        const int cb = c_first + j;
        const int sl = (long long)U * cb < iu_g;
        return p.partials + ((size_t)cb * 2 + sl) * C::kPartFloats;
      };
      constexpr int kJ = 3;  // contributors of a round
      __nv_bfloat16* o_at = p.out + row_of(at.qc, at.b, at.h) + kl;
      const int ncol = columns(at.qc, at.b);
      const int d_row = kl < DH ? kl : 0;
      float bad = 0.f;
#pragma unroll 1
      for (int f = f0; f < f0 + NF; f += 8) {
        float M[8], L[8], acc[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          M[c] = kNone;
          L[c] = acc[c] = 0.f;
        }
#pragma unroll 1
        for (int j0 = 0; j0 < n_c; j0 += kJ) {
          float4 m[kJ][2], l4[kJ][2], o[kJ][2];
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            // past the last contributor: its values once more, not used
            const float* pc = part_of(min(j0 + j, n_c - 1));
            const float4* ml = reinterpret_cast<const float4*>(pc + (size_t)NQ * DH + f);
            const float4* ov = reinterpret_cast<const float4*>(pc) + f / 4 * DH + d_row;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              m[j][v] = __ldcg(ml + v);
              l4[j][v] = __ldcg(ml + NQ / 4 + v);
              o[j][v] = __ldcg(ov + v * DH);
            }
            bad += __ldcg(pc + (size_t)NQ * DH + 2 * NQ);
          }
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            if (j0 + j >= n_c) break;
            const float mj[8] = {m[j][0].x, m[j][0].y, m[j][0].z, m[j][0].w,
                                 m[j][1].x, m[j][1].y, m[j][1].z, m[j][1].w};
            const float lj[8] = {l4[j][0].x, l4[j][0].y, l4[j][0].z, l4[j][0].w,
                                 l4[j][1].x, l4[j][1].y, l4[j][1].z, l4[j][1].w};
            const float oj[8] = {o[j][0].x, o[j][0].y, o[j][0].z, o[j][0].w,
                                 o[j][1].x, o[j][1].y, o[j][1].z, o[j][1].w};
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float mn = fmaxf(M[c], mj[c]);
              const float a = ex2_approx(M[c] - mn), w = ex2_approx(mj[c] - mn);
              L[c] = L[c] * a + w * lj[c];
              acc[c] = acc[c] * a + w * oj[c];
              M[c] = mn;
            }
          }
        }
        if (kl < DH) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (f + c < ncol)
              o_at[col_off[f + c]] = __float2bfloat16_rn(__fdividef(acc[c], L[c]));
        }
      }
      if (bad != 0.f && kl < DH)
        add_unfit<DH, FP8>(p, at.qc, at.b, at.h, s_len[at.b], s_nn[at.b], f0, f0 + NF, kl);
    }
  } else {
    // ------------------------------------------------------------ Q, finisher
    // 8 bits: the next items' rows as two e4m3 parts, each in the Q buffer its QKs will read
    // (the range's first is split by the softmax warps).  Then, for each partial of this
    // CTA: wait until the softmax warps have issued its stores, make them visible
    // device-wide, count this contributor in.  The last of an item's contributors merges
    // it, after its range.
    if constexpr (FP8) {
      Cursor cq;
      cq.init(u0, S);
      int left = T - (cq.tb - cq.t);
      for (int n = 1; left > 0; ++n) {
        const int qb = n & 1;
        cq.next_item(S);
        split_q<NQ, DH, 2>(
            static_cast<const __nv_bfloat16*>(p.q) + row_of(cq.qc, cq.b, cq.h), col_off,
            columns(cq.qc, cq.b), warp - 2, q_buf + qb * C::kQParts * C::kQPart, qsc + qb * 32,
            [&] {
              wait_while_moving(&q_empty[qb], ((uint32_t)(n >> 1) & 1u) ^ 1u, &I->done, abort_flag,
                                p.status);
            });
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&q_full[qb]);
        left -= cq.tb;
      }
    }
    if (warp == C::kFinisher) {
      if (lane == 0) {
        I->merge_u[0] = -1;
        I->merge_u[1] = -1;
        Cursor ca, cz;
        ca.init(u0, S);
        cz.init(u1 - 1, S);
#pragma unroll 1
        for (int slot = 0; slot < 2; ++slot) {
          const int iu = slot == 0 ? u0 - ca.t : u1 - 1 - cz.t;
          const int tb = slot == 0 ? ca.tb : cz.tb;
          if (slot == 1 && iu == u0 - ca.t) break;
          if (u0 <= iu && u1 >= iu + tb) continue;  // whole: the softmax warps write it
          if (!wait_while_moving(&fin_full[slot], 0u, &I->done, abort_flag, p.status)) break;
          fence_gpu();
          const int c_first = owner_of(iu, U, G), c_last = owner_of(iu + tb - 1, U, G);
          // an item that goes on behind CTA c_first's range is the only one to do so, so
          // c_first names its counter
          const unsigned prev = atomicAdd(&p.cnt[c_first], 1u);
          if (prev == (unsigned)(c_last - c_first)) {
            fence_gpu();
            p.cnt[c_first] = 0u;  // for the next call
            I->merge_u[slot] = iu;
          }
        }
      }
      __syncwarp();
      tc::named_bar_sync(5, kSmx + 32);
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tc::tmem_dealloc(tmem, ncols);
  }
}

struct TreePlan {
  int NQ, tn, gs, hs, n_qc, nk, nv, grid;
  size_t smem_bytes;
};

// Rows of an item: the smallest instance that takes them all, else chunks of 64 (of
// whole nodes).  8 bits: chunks of 32.  (At 64 the parts' columns leave TMEM room for one
// group only: 5000 cycles a tile against 2 x 2000 for two chunks of 32.)
TreePlan plan(const TreeAttnArgs& a, int num_sms) {
  TreePlan q{};
  const int g = a.Hq / a.Hkv, rows = a.T * g;
  if (a.fp8)
    q.NQ = 32;
  else
    q.NQ = rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 48 ? 48 : 64));
  q.hs = g > q.NQ ? 2 : 1;
  q.gs = (g + q.hs - 1) / q.hs;
  q.tn = q.NQ / q.gs < a.T ? q.NQ / q.gs : a.T;
  q.n_qc = (a.T + q.tn - 1) / q.tn * q.hs;
  const long long units = (long long)a.B * a.Hkv * q.n_qc * ((a.N + kKT - 1) / kKT);
  q.grid = (int)(units < num_sms ? units : num_sms);
  const size_t boxes = a.fp8 ? 1 : a.dh / 64, elt = a.fp8 ? 1 : 2;
  const size_t tile = (size_t)kKT * a.dh * elt;
  const size_t nqp = q.NQ == 48 ? 64 : q.NQ;
  size_t qbytes = a.fp8 ? (size_t)4 * q.NQ * a.dh : boxes * q.NQ * 128;
  qbytes = align_up(qbytes, 1024);
  const size_t pbytes = 2 * kKT * (a.fp8 ? 128 : nqp * 2);
  const size_t misc = Misc::kBytes + Misc::seq_bytes(a.B) +
                      (a.fp8 ? 8 * 1024 : 0);  // 8 stages of scales
  const size_t fixed = 1024 + qbytes + pbytes + misc;
  int tiles = (int)((kSmemBudget - fixed) / tile);
  if (tiles > 16) tiles = 16;
  // a V tile is held longer than a K tile: V gets the odd one
  q.nv = (tiles + 1) / 2;
  q.nk = tiles - q.nv;
  q.smem_bytes = fixed + (size_t)tiles * tile;
  return q;
}

size_t part_floats(int NQ, int dh) { return (size_t)NQ * dh + 2 * NQ + 4; }

// Raises a kernel's shared-memory limit, once a device (a bit of `done`; setting it twice
// does no harm).
cudaError_t allow_smem(const void* kern, std::atomic<unsigned long long>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBudget);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}
template <int NQ, int DH, bool FP8>
std::atomic<unsigned long long> raised{0};

template <int NQ, int DH, bool FP8>
cudaError_t launch_t(const TreePlan& q, TreeParams prm, const CUtensorMap* maps,
                     cudaStream_t stream) {
  using C = Cfg<NQ, DH, FP8>;
  auto kern = tree_tc_kernel<NQ, DH, FP8>;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), &raised<NQ, DH, FP8>);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(q.grid);
  cfg.blockDim = dim3(C::kAll);
  cfg.dynamicSmemBytes = q.smem_bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], prm);
  count_launches(1);
  return e;
}

}  // namespace

size_t tree_tc_workspace_bytes(int Hq, int Hkv, int dh, int T, int num_sms) {
  // the larger of the two cache forms
  const int rows = T * (Hq / Hkv);
  const int NQ = rows <= 32 ? 32 : (rows <= 48 ? 48 : 64);
  const size_t floats = part_floats(NQ, dh);
  return align_up((size_t)num_sms * 2 * floats * sizeof(float), 256);
}

cudaError_t launch_tree_tc(const TreeAttnArgs& a, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms > kTreeCounters) return cudaErrorInvalidValue;
  const TreePlan q = plan(a, sms);
  if (q.nk < 2 || q.nv < 2) return cudaErrorInvalidValue;
  if (tree_tc_workspace_bytes(a.Hq, a.Hkv, a.dh, a.T, sms) > a.ws_bytes) return cudaErrorInvalidValue;
  const uint64_t dh = a.dh, g = a.Hq / a.Hkv;
  CUtensorMap maps[3];
  if (!a.fp8) {
    // q [B, T, Hkv, g, dh]: box {64 dh, g heads, 1 kv head, tn nodes, 1 sequence}
    const uint64_t dims[5] = {dh, g, (uint64_t)a.Hkv, (uint64_t)a.T, (uint64_t)a.B};
    const uint64_t strides[4] = {dh * 2, g * dh * 2, (uint64_t)a.Hq * dh * 2,
                                 (uint64_t)a.T * a.Hq * dh * 2};
    const uint32_t box[5] = {64, (uint32_t)g, 1, (uint32_t)q.tn, 1};
    if (!encode_bf16_map(&maps[0], 5, a.q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_128B))
      return cudaErrorInvalidValue;
  }
  const void* src[2] = {a.k_cache, a.v_cache};
  for (int i = 0; i < 2; ++i) {
    const uint64_t elt = a.fp8 ? 1 : 2;
    const uint64_t dims[3] = {dh, (uint64_t)a.N, (uint64_t)a.B * a.Hkv};
    const uint64_t strides[2] = {dh * elt, (uint64_t)a.N * dh * elt};
    const uint32_t box[3] = {a.fp8 ? (uint32_t)a.dh : 64, kKT, 1};
    const bool ok =
        a.fp8 ? encode_u8_map(&maps[1 + i], 3, src[i], dims, strides, box,
                              a.dh == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B)
              : encode_bf16_map(&maps[1 + i], 3, src[i], dims, strides, box,
                                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    if (!ok) return cudaErrorInvalidValue;
  }
  if (a.fp8) maps[0] = maps[1];  // not read
  TreeParams prm{};
  prm.B = a.B; prm.N = a.N; prm.Hq = a.Hq; prm.Hkv = a.Hkv; prm.g = (int)g; prm.T = a.T;
  prm.n_qc = q.n_qc; prm.tn = q.tn; prm.gs = q.gs; prm.hs = q.hs; prm.nk = q.nk; prm.nv = q.nv;
  prm.keep = q.n_qc > 1;
  prm.qk_scale = kLog2e / sqrtf((float)a.dh);
  prm.q = a.q; prm.v_cache = a.v_cache; prm.k_scale = a.k_scale; prm.v_scale = a.v_scale;
  prm.cache_len = a.cache_len; prm.parent = a.parent; prm.n_nodes = a.n_nodes;
  prm.out = static_cast<__nv_bfloat16*>(a.out);
  prm.status = a.status;
  prm.cnt = a.cnt;
  prm.partials = static_cast<float*>(a.ws);
#define FDLLM_TREE_CASE(NQv, DHv, FP8v) \
  if (q.NQ == NQv && a.dh == DHv && (a.fp8 != 0) == FP8v) return launch_t<NQv, DHv, FP8v>(q, prm, maps, stream);
  FDLLM_TREE_CASE(16, 64, false)
  FDLLM_TREE_CASE(32, 64, false)
  FDLLM_TREE_CASE(48, 64, false)
  FDLLM_TREE_CASE(64, 64, false)
  FDLLM_TREE_CASE(16, 128, false)
  FDLLM_TREE_CASE(32, 128, false)
  FDLLM_TREE_CASE(48, 128, false)
  FDLLM_TREE_CASE(64, 128, false)
  FDLLM_TREE_CASE(32, 64, true)
  FDLLM_TREE_CASE(32, 128, true)
#undef FDLLM_TREE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace fdllm
