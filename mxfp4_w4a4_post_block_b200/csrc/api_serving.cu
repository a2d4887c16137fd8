// extern "C" boundary of the serving operators: few-token products with 4-bit weights, the 8-bit
// paged cache and its attention, products grouped by expert.  Argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/batq.h"
#include "kernels.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(batq_dtype t) { return t == BATQ_F32 || t == BATQ_BF16; }
size_t dtype_size(batq_dtype t) { return t == BATQ_BF16 ? 2 : 4; }
size_t round_up(size_t v, size_t m) { return (v + m - 1) / m * m; }

// Rows of `row` elements, `ld` elements apart, read or written in 16-byte pieces.
batq_status check_rows(const void* p, batq_dtype t, long long row, int ld) {
  if (ld < row) return BATQ_ERR_SHAPE;
  if (!aligned(p, 16) || ((size_t)ld * dtype_size(t)) % 16 != 0) return BATQ_ERR_ALIGNMENT;
  return BATQ_OK;
}

batq_status status_of(cudaError_t e) {
  if (e == cudaErrorInvalidValue) return BATQ_ERR_ALIGNMENT;  // a tensor map that cannot be encoded
  return e == cudaSuccess ? BATQ_OK : BATQ_ERR_CUDA;
}

// What the cache's writer and its reader both take.
batq_status check_kv8(int T, int kv_heads, int head_dim, const int* cu_dev, const int* seq_lens_dev,
                      const int* page_table_dev, int batch, int max_pages, int num_pages, int page_size,
                      const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                      const uint8_t* v_scales) {
  if (!seq_lens_dev || !page_table_dev || !k_codes || !k_scales || !v_codes || !v_scales) return BATQ_ERR_INVALID_ARG;
  if (T < 1 || kv_heads < 1 || batch < 1 || max_pages < 1 || num_pages < 1) return BATQ_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return BATQ_ERR_SHAPE;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return BATQ_ERR_SHAPE;
  if (kv_heads > 1024 || batch > 65535) return BATQ_ERR_SHAPE;
  // Token numbers stay 32-bit for some tiles of a look ahead behind the longest sequence.
  if ((long long)max_pages * page_size > (1LL << 31) - 16384) return BATQ_ERR_SHAPE;
  if ((long long)num_pages * kv_heads * page_size >= (1LL << 31)) return BATQ_ERR_SHAPE;  // cache rows
  if (!cu_dev && T < batch) return BATQ_ERR_SHAPE;
  if (!aligned(seq_lens_dev, 4) || !aligned(page_table_dev, 4) || (cu_dev && !aligned(cu_dev, 4)) ||
      !aligned(k_codes, 16) || !aligned(v_codes, 16))
    return BATQ_ERR_ALIGNMENT;
  return BATQ_OK;
}

batq_status check_attn_shape(int max_q_len, int q_heads, int kv_heads, int head_dim) {
  if (max_q_len < 1 || q_heads < 1 || kv_heads < 1 || kv_heads > 1024 || q_heads % kv_heads != 0)
    return BATQ_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return BATQ_ERR_SHAPE;
  if ((long long)max_q_len * q_heads >= (1LL << 31)) return BATQ_ERR_SHAPE;
  return BATQ_OK;
}

batq_status check_experts(const uint8_t* w_codes, const uint8_t* w_scales, const int* offsets_dev, int E, int T,
                          int M, int N, batq_dtype out_dtype, const void* out, int ldo) {
  if (!w_codes || !w_scales || !offsets_dev || !out || !dtype_ok(out_dtype)) return BATQ_ERR_INVALID_ARG;
  if (E < 1 || E > batq::kMaxExperts || T < 1 || N < 64 || N % 64 != 0 || M < 16 || M % 16 != 0)
    return BATQ_ERR_SHAPE;
  // Rows, tiles and scale rows stay inside 32-bit arithmetic.
  if ((long long)T * (N / 32) >= (1LL << 31) || (long long)E * round_up(M, 128) * (N / 32) >= (1LL << 31))
    return BATQ_ERR_SHAPE;
  if (((long long)E + T / 256) * ((M + 255) / 256) >= (1LL << 31)) return BATQ_ERR_SHAPE;
  batq_status st = check_rows(out, out_dtype, M, ldo);
  if (st != BATQ_OK) return st;
  if (!aligned(w_codes, 16) || !aligned(w_scales, 16) || !aligned(offsets_dev, 4)) return BATQ_ERR_ALIGNMENT;
  return BATQ_OK;
}

}  // namespace

extern "C" {

batq_status batq_linear_w4a16(const void* X, batq_dtype x_dtype, int S, int N, int ldx, const float* A_host,
                              const float* B_dev, batq_w4_format w_format, const uint8_t* w_codes,
                              const uint8_t* w_scales, const float* w_gs_dev, int M, batq_dtype out_dtype, void* out,
                              int ldo, void* stream) {
  if (!X || !w_codes || !w_scales || !out || !dtype_ok(x_dtype) || !dtype_ok(out_dtype)) return BATQ_ERR_INVALID_ARG;
  if ((A_host == nullptr) != (B_dev == nullptr)) return BATQ_ERR_INVALID_ARG;
  if (w_format != BATQ_W4_MXFP4 && w_format != BATQ_W4_NVFP4) return BATQ_ERR_INVALID_ARG;
  if (w_gs_dev && w_format != BATQ_W4_NVFP4) return BATQ_ERR_INVALID_ARG;
  if (S < 1 || S > batq::kMaxW4A16Tokens || N < 64 || N % 64 != 0 ||
      N > (w_format == BATQ_W4_NVFP4 ? batq::kMaxW4A16NvN : batq::kMaxW4A16N))
    return BATQ_ERR_SHAPE;
  if (M < 16 || M % 16 != 0 || (long long)M * (N / 32) >= (1LL << 31)) return BATQ_ERR_SHAPE;
  batq_status st = check_rows(X, x_dtype, N, ldx);
  if (st != BATQ_OK) return st;
  st = check_rows(out, out_dtype, M, ldo);
  if (st != BATQ_OK) return st;
  if (!aligned(w_codes, 16) || !aligned(w_scales, 16) || (B_dev && !aligned(B_dev, 16)) ||
      (w_gs_dev && !aligned(w_gs_dev, 4)))
    return BATQ_ERR_ALIGNMENT;
  st = static_cast<batq_status>(batq::arch_status());
  if (st != BATQ_OK) return st;
  batq::LinearW4A16Launch L = {};
  L.X = X;
  L.x_bf16 = x_dtype == BATQ_BF16;
  L.S = S;
  L.N = N;
  L.ldx = ldx;
  L.transform = A_host != nullptr;
  if (A_host) std::memcpy(L.A, A_host, sizeof(L.A));
  L.B = B_dev;
  L.nvfp4 = w_format == BATQ_W4_NVFP4;
  L.w_codes = w_codes;
  L.w_scales = w_scales;
  L.w_gs = w_gs_dev;
  L.M = M;
  L.out_bf16 = out_dtype == BATQ_BF16;
  L.out = out;
  L.ldo = ldo;
  L.err = batq::device_error_word();
  return status_of(batq::launch_linear_w4a16(L, static_cast<cudaStream_t>(stream)));
}

batq_status batq_kv8_append(const void* K, const void* V, batq_dtype dtype, int T, int kv_heads, int head_dim, int ldk,
                            int ldv, const int* cu_new_dev, const int* seq_lens_dev, const int* page_table_dev,
                            int batch, int max_pages, int num_pages, int page_size, uint8_t* k_codes,
                            uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales, void* stream) {
  if (!K || !V || !dtype_ok(dtype)) return BATQ_ERR_INVALID_ARG;
  batq_status st = check_kv8(T, kv_heads, head_dim, cu_new_dev, seq_lens_dev, page_table_dev, batch, max_pages,
                             num_pages, page_size, k_codes, k_scales, v_codes, v_scales);
  if (st != BATQ_OK) return st;
  st = check_rows(K, dtype, (long long)kv_heads * head_dim, ldk);
  if (st != BATQ_OK) return st;
  st = check_rows(V, dtype, (long long)kv_heads * head_dim, ldv);
  if (st != BATQ_OK) return st;
  st = static_cast<batq_status>(batq::arch_status());
  if (st != BATQ_OK) return st;
  batq::Kv8AppendLaunch L = {K,       V,         dtype == BATQ_BF16, T,         kv_heads, head_dim, ldk,
                             ldv,     cu_new_dev, seq_lens_dev,       page_table_dev, batch, max_pages, num_pages,
                             page_size, k_codes,  k_scales,           v_codes,   v_scales};
  return status_of(batq::launch_kv8_append(L, static_cast<cudaStream_t>(stream)));
}

batq_status batq_attn_kv8_workspace_size(int max_q_len, int q_heads, int kv_heads, int head_dim, size_t* bytes) {
  if (!bytes) return BATQ_ERR_INVALID_ARG;
  batq_status st = check_attn_shape(max_q_len, q_heads, kv_heads, head_dim);
  if (st != BATQ_OK) return st;
  *bytes = batq::attn_kv8_workspace_bytes(max_q_len, q_heads, kv_heads, head_dim);
  return BATQ_OK;
}

batq_status batq_attn_kv8(const void* Q, batq_dtype q_dtype, int T, int ldq, int q_heads, int kv_heads, int head_dim,
                          const int* cu_q_dev, const int* seq_lens_dev, const int* page_table_dev, int batch,
                          int max_pages, int num_pages, int page_size, const uint8_t* k_codes,
                          const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales,
                          float softmax_scale, int max_q_len, void* workspace, size_t workspace_bytes,
                          batq_dtype out_dtype, void* out, int ldo, float* lse, void* stream) {
  if (!Q || !out || !workspace || !dtype_ok(q_dtype) || !dtype_ok(out_dtype) || !std::isfinite(softmax_scale))
    return BATQ_ERR_INVALID_ARG;
  batq_status st = check_attn_shape(max_q_len, q_heads, kv_heads, head_dim);
  if (st != BATQ_OK) return st;
  st = check_kv8(T, kv_heads, head_dim, cu_q_dev, seq_lens_dev, page_table_dev, batch, max_pages, num_pages, page_size,
                 k_codes, k_scales, v_codes, v_scales);
  if (st != BATQ_OK) return st;
  // Work units (blocks of 64 keys or more of 8 rows or more) stay inside 32-bit arithmetic.
  if ((long long)batch * kv_heads * (((long long)max_q_len * (q_heads / kv_heads) + 7) / 8) >
      (1LL << 31) / (((long long)max_pages * page_size + 63) / 64 + 1))
    return BATQ_ERR_SHAPE;
  // No sequence has more queries than there are rows, or than one without cu: what max_q_len says beyond is not paid for.
  const int most_q = cu_q_dev ? (max_q_len < T ? max_q_len : T) : 1;
  if ((long long)most_q * q_heads >= (1LL << 31) - 8) return BATQ_ERR_SHAPE;  // rows of the join's grid
  const long long row = (long long)q_heads * head_dim;
  st = check_rows(Q, q_dtype, row, ldq);
  if (st != BATQ_OK) return st;
  st = check_rows(out, out_dtype, row, ldo);
  if (st != BATQ_OK) return st;
  if (!aligned(workspace, 16) || (lse && !aligned(lse, 4))) return BATQ_ERR_ALIGNMENT;
  if (workspace_bytes < batq::attn_kv8_workspace_bytes(max_q_len, q_heads, kv_heads, head_dim))
    return BATQ_ERR_WORKSPACE;
  st = static_cast<batq_status>(batq::arch_status());
  if (st != BATQ_OK) return st;
  batq::AttnKv8Launch L = {};
  L.Q = Q;
  L.q_bf16 = q_dtype == BATQ_BF16;
  L.T = T;
  L.ldq = ldq;
  L.q_heads = q_heads;
  L.kv_heads = kv_heads;
  L.head_dim = head_dim;
  L.cu_q = cu_q_dev;
  L.seq_lens = seq_lens_dev;
  L.page_table = page_table_dev;
  L.batch = batch;
  L.max_pages = max_pages;
  L.num_pages = num_pages;
  L.page_size = page_size;
  L.k_codes = k_codes;
  L.k_scales = k_scales;
  L.v_codes = v_codes;
  L.v_scales = v_scales;
  L.softmax_scale = softmax_scale;
  L.max_q_len = most_q;
  L.workspace = static_cast<float*>(workspace);
  L.out_bf16 = out_dtype == BATQ_BF16;
  L.out = out;
  L.ldo = ldo;
  L.lse = lse;
  L.err = batq::device_error_word();
  return status_of(batq::launch_attn_kv8(L, static_cast<cudaStream_t>(stream)));
}

batq_status batq_gemm_mxfp4_experts(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* w_codes,
                                    const uint8_t* w_scales, const int* expert_offsets_dev, int E, int T, int M, int N,
                                    batq_dtype out_dtype, void* out, int ldo, void* stream) {
  if (!a_codes || !a_scales) return BATQ_ERR_INVALID_ARG;
  batq_status st = check_experts(w_codes, w_scales, expert_offsets_dev, E, T, M, N, out_dtype, out, ldo);
  if (st != BATQ_OK) return st;
  if (!aligned(a_codes, 16) || !aligned(a_scales, 16)) return BATQ_ERR_ALIGNMENT;
  st = static_cast<batq_status>(batq::arch_status());
  if (st != BATQ_OK) return st;
  batq::ExpertsLaunch L = {a_codes, a_scales, w_codes, w_scales, expert_offsets_dev, E, T, M, N,
                           out_dtype == BATQ_BF16, out, ldo, batq::device_error_word()};
  return status_of(batq::launch_gemm_experts(L, static_cast<cudaStream_t>(stream)));
}

batq_status batq_linear_experts_workspace_size(int T, int N, size_t* bytes) {
  if (!bytes) return BATQ_ERR_INVALID_ARG;
  size_t codes = 0, scales = 0;
  batq_status st = batq_act_buffer_sizes(T, N, BATQ_SCALES_LINEAR, &codes, &scales);
  if (st != BATQ_OK) return st;
  *bytes = round_up(codes, 256) + round_up(scales, 256);
  return BATQ_OK;
}

batq_status batq_linear_experts(const void* X, batq_dtype x_dtype, int T, int N, int ldx, const float* A_host,
                                const float* B_dev, const float* ratios_dev, const uint8_t* w_codes,
                                const uint8_t* w_scales, const int* expert_offsets_dev, int E, int M, void* workspace,
                                size_t workspace_bytes, batq_dtype out_dtype, void* out, int ldo, void* stream) {
  if (!workspace) return BATQ_ERR_INVALID_ARG;
  size_t need = 0;
  batq_status st = batq_linear_experts_workspace_size(T, N, &need);
  if (st != BATQ_OK) return st;
  if (workspace_bytes < need) return BATQ_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return BATQ_ERR_ALIGNMENT;
  st = check_experts(w_codes, w_scales, expert_offsets_dev, E, T, M, N, out_dtype, out, ldo);
  if (st != BATQ_OK) return st;
  uint8_t* codes = static_cast<uint8_t*>(workspace);
  uint8_t* scales = codes + round_up((size_t)T * (N / 2), 256);
  st = batq_quant_act(X, x_dtype, T, N, ldx, A_host, B_dev, ratios_dev, codes, scales, BATQ_SCALES_LINEAR, nullptr,
                      stream);
  if (st != BATQ_OK) return st;
  return batq_gemm_mxfp4_experts(codes, scales, w_codes, w_scales, expert_offsets_dev, E, T, M, N, out_dtype, out, ldo,
                                 stream);
}

}  // extern "C"
