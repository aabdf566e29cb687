// C ABI of the calls for drafted tokens: 8-bit cache rows, tree attention and
// sampled verification.  The operations are defined in include/fdllm.h.
#include "api_util.h"
#include "common.cuh"
#include "kernels.h"

using namespace fdllm;

namespace {

constexpr long long kMaxInt = (1ll << 31) - 1;

fdllm_status check_rows(int B, int N, int H, int dh, int R, int dtype) {
  if (B < 0 || N < 1 || H < 1 || R < 0) return FDLLM_ERR_INVALID_ARG;
  if (dtype != FDLLM_F32 && dtype != FDLLM_BF16) return FDLLM_ERR_UNSUPPORTED;
  if (dh != 64 && dh != 128) return FDLLM_ERR_UNSUPPORTED;
  // units are counted in 32 bits: CTAs (at most one a row), (row, head) pairs of a block
  if ((long long)B * R > kMaxInt || H > (1 << 20) || (long long)B * N > (1ll << 31))
    return FDLLM_ERR_UNSUPPORTED;
  return FDLLM_OK;
}

fdllm_status check_tree(int B, int N, int Hq, int Hkv, int dh, int T, int dtype) {
  if (B < 0 || N < 1 || Hkv < 1 || Hq < Hkv || T < 0) return FDLLM_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return FDLLM_ERR_INVALID_ARG;
  if (dtype != FDLLM_F32 && dtype != FDLLM_BF16) return FDLLM_ERR_UNSUPPORTED;
  if (dh != 64 && dh != 128) return FDLLM_ERR_UNSUPPORTED;
  if (T > FDLLM_MAX_TREE_NODES || B > FDLLM_MAX_TREE_SEQS || Hq / Hkv > 64 || Hq > 4096)
    return FDLLM_ERR_UNSUPPORTED;
  if ((long long)B * N > (1ll << 31) || N > (1 << 30)) return FDLLM_ERR_UNSUPPORTED;
  // work units (chunk of at most 32 rows, sequence, kv head, 128 slots)
  // are counted in 32 bits
  const int g = Hq / Hkv, tn = g < 32 ? 32 / g : 1, chunks = (T + tn - 1) / tn * (g > 32 ? 2 : 1);
  if ((long long)B * Hkv * ((N + 127) / 128) * chunks > (1ll << 30)) return FDLLM_ERR_UNSUPPORTED;
  return FDLLM_OK;
}

fdllm_status check_draft(int B, int T, int V, int most) {
  if (B < 0 || T < 0 || V < 1) return FDLLM_ERR_INVALID_ARG;
  if (T > most || B > kMaxVerifySeqs || V > (1 << 30)) return FDLLM_ERR_UNSUPPORTED;
  return FDLLM_OK;
}

// Workspaces: [header | counters, zero between calls | what a call leaves behind].  The
// counters lie at the same place for attention and verification, whatever the shapes are:
// neither writes where the other expects zeros.
constexpr size_t kCountersOff = kWsHeaderBytes;
constexpr size_t kScratchOff = kCountersOff + kMaxVerifySeqs * sizeof(unsigned);

size_t draft_verify_bytes(int B, int V) { return kScratchOff + draft_verify_parts_bytes(B, V); }

void set_verify_ws(DraftVerifyArgs* a, void* ws) {
  a->status = reinterpret_cast<int*>(ws);
  a->seq_cnt = reinterpret_cast<unsigned*>(ws_at(ws, kCountersOff));
  a->parts = reinterpret_cast<double*>(ws_at(ws, kScratchOff));
}

fdllm_status run_tree(const TreeAttnArgs& args, void* workspace, size_t workspace_bytes,
                      void* stream) {
  TreeAttnArgs a = args;
  fdllm_status st = check_tree(a.B, a.N, a.Hq, a.Hkv, a.dh, a.T, a.dtype);
  if (st != FDLLM_OK) return st;
  if (a.fp8 && a.dtype != FDLLM_BF16) return FDLLM_ERR_UNSUPPORTED;
  const size_t need = fdllm_tree_attend_workspace_bytes(a.B, a.N, a.Hq, a.Hkv, a.dh, a.T, a.dtype);
  if ((st = check_ws(workspace, workspace_bytes, need)) != FDLLM_OK) return st;
  if (a.B * a.T == 0) return FDLLM_OK;
  if (!all_aligned({a.q, a.k_cache, a.v_cache, a.cache_len, a.out})) return FDLLM_ERR_INVALID_ARG;
  if (a.fp8 && !all_aligned({a.k_scale, a.v_scale})) return FDLLM_ERR_INVALID_ARG;
  if ((a.parent && !aligned16(a.parent)) || (a.n_nodes && !aligned16(a.n_nodes)))
    return FDLLM_ERR_INVALID_ARG;
  a.status = reinterpret_cast<int*>(workspace);
  if (a.dtype != FDLLM_F32) {
    a.cnt = reinterpret_cast<unsigned*>(ws_at(workspace, kCountersOff));
    a.ws = ws_at(workspace, kScratchOff);
    a.ws_bytes = need - kScratchOff;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return from_cuda(tree_simt_takes(a) ? launch_tree_simt(a, s) : launch_tree_tc(a, s));
}

}  // namespace

extern "C" {

size_t fdllm_cache_fp8_workspace_bytes(int B, int R) {
  return B < 0 || R < 0 ? 0 : kWsHeaderBytes;
}

fdllm_status fdllm_cache_write_fp8(int B, int N, int H, int dh, int R, int dtype,
                                   const void* k_rows, const void* v_rows, const int32_t* pos,
                                   void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("fdllm_cache_write_fp8");
  fdllm_status st = check_rows(B, N, H, dh, R, dtype);
  if (st != FDLLM_OK) return st;
  if ((st = check_ws(workspace, workspace_bytes, kWsHeaderBytes)) != FDLLM_OK) return st;
  if (B == 0 || R == 0) return FDLLM_OK;
  if (!all_aligned({k_rows, v_rows, pos, k_cache, v_cache, k_scale, v_scale}))
    return FDLLM_ERR_INVALID_ARG;
  CacheFp8Args a{};
  a.B = B; a.N = N; a.H = H; a.dh = dh; a.R = R; a.dtype = dtype;
  a.pos = pos;
  a.k_rows = const_cast<void*>(k_rows); a.v_rows = const_cast<void*>(v_rows);
  a.k_cache = static_cast<uint8_t*>(k_cache); a.v_cache = static_cast<uint8_t*>(v_cache);
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.status = reinterpret_cast<int*>(workspace);
  return from_cuda(launch_cache_write_fp8(a, static_cast<cudaStream_t>(stream)));
}

fdllm_status fdllm_cache_read_fp8(int B, int N, int H, int dh, int R, int dtype,
                                  const int32_t* pos, const void* k_cache, const void* v_cache,
                                  const float* k_scale, const float* v_scale, void* k_rows,
                                  void* v_rows, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  NvtxRange nvtx_range("fdllm_cache_read_fp8");
  fdllm_status st = check_rows(B, N, H, dh, R, dtype);
  if (st != FDLLM_OK) return st;
  if ((st = check_ws(workspace, workspace_bytes, kWsHeaderBytes)) != FDLLM_OK) return st;
  if (B == 0 || R == 0) return FDLLM_OK;
  if (!all_aligned({k_rows, v_rows, pos, k_cache, v_cache, k_scale, v_scale}))
    return FDLLM_ERR_INVALID_ARG;
  CacheFp8Args a{};
  a.B = B; a.N = N; a.H = H; a.dh = dh; a.R = R; a.dtype = dtype;
  a.pos = pos;
  a.k_rows = k_rows; a.v_rows = v_rows;
  a.k_cache = static_cast<uint8_t*>(const_cast<void*>(k_cache));
  a.v_cache = static_cast<uint8_t*>(const_cast<void*>(v_cache));
  a.k_scale = const_cast<float*>(k_scale); a.v_scale = const_cast<float*>(v_scale);
  a.status = reinterpret_cast<int*>(workspace);
  return from_cuda(launch_cache_read_fp8(a, static_cast<cudaStream_t>(stream)));
}

size_t fdllm_tree_attend_workspace_bytes(int B, int N, int Hq, int Hkv, int dh, int T, int dtype) {
  if (check_tree(B, N, Hq, Hkv, dh, T, dtype) != FDLLM_OK) return 0;
  if (dtype == FDLLM_F32) return kWsHeaderBytes;
  return kScratchOff + tree_tc_workspace_bytes(Hq, Hkv, dh, T, device_sm_count());
}

fdllm_status fdllm_tree_attend(int B, int N, int Hq, int Hkv, int dh, int T, int dtype,
                               const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* cache_len, const int32_t* parent,
                               const int32_t* n_nodes, void* out, void* workspace,
                               size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("fdllm_tree_attend");
  TreeAttnArgs a{};
  a.B = B; a.N = N; a.Hq = Hq; a.Hkv = Hkv; a.dh = dh; a.T = T; a.dtype = dtype;
  a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
  a.cache_len = cache_len; a.parent = parent; a.n_nodes = n_nodes; a.out = out;
  return run_tree(a, workspace, workspace_bytes, stream);
}

fdllm_status fdllm_tree_attend_fp8(int B, int N, int Hq, int Hkv, int dh, int T, int dtype,
                                   const void* q, const void* k_cache, const void* v_cache,
                                   const float* k_scale, const float* v_scale,
                                   const int32_t* cache_len, const int32_t* parent,
                                   const int32_t* n_nodes, void* out, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("fdllm_tree_attend_fp8");
  TreeAttnArgs a{};
  a.B = B; a.N = N; a.Hq = Hq; a.Hkv = Hkv; a.dh = dh; a.T = T; a.dtype = dtype;
  a.fp8 = 1;
  a.q = q; a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
  a.cache_len = cache_len; a.parent = parent; a.n_nodes = n_nodes; a.out = out;
  return run_tree(a, workspace, workspace_bytes, stream);
}

size_t fdllm_draft_verify_workspace_bytes(int B, int T, int V) {
  if (check_draft(B, T, V, FDLLM_MAX_CHAIN) != FDLLM_OK) return 0;
  return draft_verify_bytes(B, V);
}

fdllm_status fdllm_chain_verify(int B, int T, int V, const float* target, const float* draft,
                                const int32_t* tok, const int32_t* n_draft, const float* u,
                                const float* r, int32_t* n_accept, int32_t* next_tok,
                                void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("fdllm_chain_verify");
  fdllm_status st = check_draft(B, T, V, FDLLM_MAX_CHAIN);
  if (st != FDLLM_OK) return st;
  if ((st = check_ws(workspace, workspace_bytes, draft_verify_bytes(B, V))) != FDLLM_OK) return st;
  if (B == 0) return FDLLM_OK;
  if (!all_aligned({target, r, n_accept, next_tok})) return FDLLM_ERR_INVALID_ARG;
  if (T > 0 && !all_aligned({draft, tok, u})) return FDLLM_ERR_INVALID_ARG;
  if (n_draft && !aligned16(n_draft)) return FDLLM_ERR_INVALID_ARG;
  DraftVerifyArgs a{};
  a.B = B; a.T = T; a.V = V;
  a.target = target; a.draft = draft; a.tok = tok; a.count = n_draft; a.u = u; a.r = r;
  a.n_accept = n_accept; a.next_tok = next_tok;
  set_verify_ws(&a, workspace);
  return from_cuda(launch_chain_verify(a, static_cast<cudaStream_t>(stream)));
}

fdllm_status fdllm_tree_verify(int B, int T, int V, const float* target, const int32_t* tok,
                               const int32_t* parent, const int32_t* n_nodes, const float* u,
                               const float* r, int32_t* path, int32_t* n_accept,
                               int32_t* next_tok, void* workspace, size_t workspace_bytes,
                               void* stream) {
  NvtxRange nvtx_range("fdllm_tree_verify");
  fdllm_status st = check_draft(B, T, V, FDLLM_MAX_TREE_NODES);
  if (st != FDLLM_OK) return st;
  if (T < 1) return FDLLM_ERR_INVALID_ARG;
  if ((st = check_ws(workspace, workspace_bytes, draft_verify_bytes(B, V))) != FDLLM_OK) return st;
  if (B == 0) return FDLLM_OK;
  if (!all_aligned({target, tok, parent, u, r, path, n_accept, next_tok}))
    return FDLLM_ERR_INVALID_ARG;
  if (n_nodes && !aligned16(n_nodes)) return FDLLM_ERR_INVALID_ARG;
  DraftVerifyArgs a{};
  a.B = B; a.T = T; a.V = V;
  a.target = target; a.tok = tok; a.parent = parent; a.count = n_nodes; a.u = u; a.r = r;
  a.path = path; a.n_accept = n_accept; a.next_tok = next_tok;
  set_verify_ws(&a, workspace);
  return from_cuda(launch_tree_verify(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
