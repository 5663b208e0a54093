// api.cu -- the C ABI of include/mx.h: argument, shape and alignment checks
// on the host, then one asynchronous launch on the caller's stream.
//
// The pages' interface (WWDC26 session 330, 3:53 / 4:48 listings): a quantized
// tensor is one object carrying a data plane and a scale plane, and creating
// one reports failure through a status rather than by crashing; the matmul
// takes two such tensors and a plain output with no transposes.  Here that is
// the mx_tensor struct plus mx_status codes.
#include <cstdint>
#include <cstring>

#include "mx.h"
#include "common.cuh"
#include "kv_common.cuh"

namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The library ships sm_103a code only: require compute capability 10.3.
mx_status check_device() {
  static int ok_cache[64] = {};   // 0 unknown, 1 ok, 2 unsupported
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MX_ERR_CUDA;
  if (dev < 64 && ok_cache[dev]) return ok_cache[dev] == 1 ? MX_OK : MX_ERR_UNSUPPORTED;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return MX_ERR_CUDA;
  const bool ok = (major == 10 && minor == 3);
  if (dev < 64) ok_cache[dev] = ok ? 1 : 2;
  return ok ? MX_OK : MX_ERR_UNSUPPORTED;
}

mx_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MX_OK : MX_ERR_CUDA; }

bool is_int_fmt(int32_t fmt) {
  return fmt == MX_FMT_INT8 || fmt == MX_FMT_INT4 || fmt == MX_FMT_INT2;
}

// A and B of one product: equal K; an E2M1 operand beside an 8-bit one is
// unpacked by TMA, which needs K % 128 == 0 and a 32-byte aligned plane.
mx_status check_pair(const mx_tensor* A, const mx_tensor* B) {
  // the tensor cores have no block-scaled integer kind: integer tensors are
  // B operands of gemm_dequant only
  if (is_int_fmt(A->fmt) || is_int_fmt(B->fmt)) return MX_ERR_INVALID_ARG;
  if (A->K != B->K) return MX_ERR_SHAPE;
  if ((A->fmt == MX_FMT_E2M1) == (B->fmt == MX_FMT_E2M1)) return MX_OK;
  if (A->outer == 0 || B->outer == 0 || A->K == 0) return MX_OK;
  if (A->K % 128) return MX_ERR_SHAPE;
  const mx_tensor* f4 = (A->fmt == MX_FMT_E2M1) ? A : B;
  if (reinterpret_cast<uintptr_t>(f4->data) % 32) return MX_ERR_ALIGN;
  return MX_OK;
}

mx_status check_tensor(const mx_tensor* t) {
  if (!t) return MX_ERR_INVALID_ARG;
  if (t->fmt < MX_FMT_E4M3 || t->fmt > MX_FMT_INT2) return MX_ERR_INVALID_ARG;
  if (t->outer < 0 || t->K < 0 || t->outer > kMaxDim || t->K > kMaxDim) return MX_ERR_SHAPE;
  if (t->K % 32) return MX_ERR_SHAPE;
  if (t->outer > 0 && t->K > 0) {
    if (!t->data || !t->scales) return MX_ERR_INVALID_ARG;
    if (!aligned16(t->data) || !aligned16(t->scales)) return MX_ERR_ALIGN;
  }
  return MX_OK;
}

// The optional epilogue argument: NULL means none.  The bias must be
// 16-byte aligned (it is read as float4).
mx_status epilogue_from(const mx_epilogue* epi, mxk::Epilogue* out) {
  *out = mxk::Epilogue{};
  if (!epi) return MX_OK;
  if (epi->act != MX_ACT_NONE && epi->act != MX_ACT_GELU && epi->act != MX_ACT_GELU_TANH)
    return MX_ERR_INVALID_ARG;
  if (epi->bias && !aligned16(epi->bias)) return MX_ERR_ALIGN;
  out->bias = epi->bias;
  out->act = epi->act;
  return MX_OK;
}

bool has_work(const mxk::Epilogue& e) { return e.bias != nullptr || e.act != MX_ACT_NONE; }

// mx_gemm, mx_gemm_splitk and mx_gemm_fused: checks, then one launch.
mx_status mx_product(const mx_tensor* A, const mx_tensor* B, const mx_epilogue* epi, void* C,
                     int32_t c_dtype, int64_t ldc, void* ws, size_t ws_bytes, void* stream) {
  mx_status s;
  if ((s = check_tensor(A)) != MX_OK) return s;
  if ((s = check_tensor(B)) != MX_OK) return s;
  if ((s = check_pair(A, B)) != MX_OK) return s;
  if (c_dtype != MX_DT_F32 && c_dtype != MX_DT_BF16) return MX_ERR_INVALID_ARG;
  mxk::Epilogue e;
  if ((s = epilogue_from(epi, &e)) != MX_OK) return s;
  const int64_t M = A->outer, N = B->outer, K = A->K;
  if (M == 0 || N == 0) return MX_OK;
  if (!C) return MX_ERR_INVALID_ARG;
  const int64_t eb = (c_dtype == MX_DT_BF16) ? 2 : 4;
  if (ldc < N || (ldc * eb) % 16) return MX_ERR_SHAPE;
  if (!aligned16(C)) return MX_ERR_ALIGN;
  if (K == 0 && has_work(e)) return MX_ERR_SHAPE;
  if ((s = check_device()) != MX_OK) return s;
  return from_cuda(mxk::launch_gemm_mx(A->fmt, B->fmt, A->data, A->scales, B->data, B->scales,
                                       C, c_dtype, ldc, M, N, K, ws, ws_bytes, e,
                                       static_cast<cudaStream_t>(stream)));
}

// gemm_f16, gemm_f16_splitk and gemm_f16_fused.
mx_status f16_product(const void* A, const void* B, const mx_epilogue* epi, float* C,
                      int32_t ab_dtype, int64_t M, int64_t N, int64_t K, int64_t lda,
                      int64_t ldb, int64_t ldc, void* ws, size_t ws_bytes, void* stream) {
  if (ab_dtype != MX_DT_F16 && ab_dtype != MX_DT_BF16) return MX_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
    return MX_ERR_SHAPE;
  mxk::Epilogue e;
  mx_status s = epilogue_from(epi, &e);
  if (s != MX_OK) return s;
  if (M == 0 || N == 0) return MX_OK;
  if (!C) return MX_ERR_INVALID_ARG;
  if (ldc < N || ldc % 4) return MX_ERR_SHAPE;
  if (!aligned16(C)) return MX_ERR_ALIGN;
  if (K > 0) {
    if (!A || !B) return MX_ERR_INVALID_ARG;
    if (lda < K || ldb < N || lda % 8 || ldb % 8) return MX_ERR_SHAPE;
    if (!aligned16(A) || !aligned16(B)) return MX_ERR_ALIGN;
  } else if (has_work(e)) {
    return MX_ERR_SHAPE;
  }
  if ((s = check_device()) != MX_OK) return s;
  return from_cuda(mxk::launch_gemm_f16(ab_dtype, A, B, C, M, N, K, lda, ldb, ldc, ws,
                                        ws_bytes, e, static_cast<cudaStream_t>(stream)));
}

}  // namespace

#pragma GCC visibility push(default)
extern "C" {

size_t mx_data_bytes(int32_t fmt, int64_t outer, int64_t K) {
  if (outer < 0 || K < 0 || K % 32) return 0;
  if (fmt < MX_FMT_E4M3 || fmt > MX_FMT_INT2) return 0;
  return static_cast<size_t>(outer) * static_cast<size_t>(K) *
         static_cast<size_t>(mxk::code_bits(fmt)) / 8;
}

size_t mx_scale_bytes(int64_t outer, int64_t K) {
  if (outer < 0 || K < 0 || K % 32) return 0;
  return static_cast<size_t>(mxk::sf_row_atoms(outer)) *
         static_cast<size_t>(mxk::sf_k_atoms(K)) * mxk::SF_ATOM_BYTES;
}

mx_status mx_quantize(const float* src, int64_t ld, int32_t src_layout, const mx_tensor* out,
                      void* stream) {
  mx_status s = check_tensor(out);
  if (s != MX_OK) return s;
  if (src_layout != MX_SRC_K_CONTIGUOUS && src_layout != MX_SRC_K_STRIDED)
    return MX_ERR_INVALID_ARG;
  if (out->outer == 0 || out->K == 0) return MX_OK;
  if (!src) return MX_ERR_INVALID_ARG;
  const int64_t inner = (src_layout == MX_SRC_K_CONTIGUOUS) ? out->K : out->outer;
  if (ld < inner || ld % 4) return MX_ERR_SHAPE;
  if (!aligned16(src)) return MX_ERR_ALIGN;
  // grid limits: 65535 CTAs along the second grid dimension
  const int64_t ra = mxk::sf_row_atoms(out->outer), ka = mxk::sf_k_atoms(out->K);
  if ((src_layout == MX_SRC_K_CONTIGUOUS ? ra : ka) > 65535) return MX_ERR_SHAPE;
  if ((s = check_device()) != MX_OK) return s;
  return from_cuda(mxk::launch_quantize(src, ld, src_layout == MX_SRC_K_STRIDED, out->fmt,
                                        out->outer, out->K, out->data, out->scales,
                                        static_cast<cudaStream_t>(stream)));
}

mx_status mx_gemm(const mx_tensor* A, const mx_tensor* B, void* C, int32_t c_dtype,
                  int64_t ldc, void* stream) {
  return mx_product(A, B, nullptr, C, c_dtype, ldc, nullptr, 0, stream);
}

size_t mx_gemm_workspace_bytes(int32_t fmt, int64_t M, int64_t N, int64_t K) {
  if (fmt != MX_FMT_E4M3 && fmt != MX_FMT_E5M2 && fmt != MX_FMT_E2M1) return 0;
  if (M <= 0 || N <= 0 || K <= 0 || K % 32 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
    return 0;
  if (check_device() != MX_OK) return 0;
  return mxk::gemm_workspace_bytes(fmt, M, N, K);
}

mx_status mx_gemm_splitk(const mx_tensor* A, const mx_tensor* B, void* C, int32_t c_dtype,
                         int64_t ldc, void* workspace, size_t workspace_bytes, void* stream) {
  if (workspace && !aligned16(workspace)) return MX_ERR_ALIGN;
  return mx_product(A, B, nullptr, C, c_dtype, ldc, workspace, workspace_bytes, stream);
}

mx_status mx_gemm_fused(const mx_tensor* A, const mx_tensor* B, const mx_epilogue* epi,
                        void* C, int32_t c_dtype, int64_t ldc, void* stream) {
  return mx_product(A, B, epi, C, c_dtype, ldc, nullptr, 0, stream);
}

mx_status mx_gemm_fused_quantize(const mx_tensor* A, const mx_tensor* B,
                                 const mx_epilogue* epi, const mx_tensor* C, void* stream) {
  mx_status s;
  if ((s = check_tensor(A)) != MX_OK) return s;
  if ((s = check_tensor(B)) != MX_OK) return s;
  if ((s = check_pair(A, B)) != MX_OK) return s;
  if ((s = check_tensor(C)) != MX_OK) return s;
  if (is_int_fmt(C->fmt)) return MX_ERR_INVALID_ARG;
  const int64_t M = A->outer, N = B->outer, K = A->K;
  if (C->outer != M || C->K != N) return MX_ERR_SHAPE;
  mxk::Epilogue e;
  if ((s = epilogue_from(epi, &e)) != MX_OK) return s;
  if (M == 0 || N == 0) return MX_OK;
  if (K == 0) return MX_ERR_SHAPE;
  if ((s = check_device()) != MX_OK) return s;
  e.q_fmt = C->fmt;
  e.q_sf = C->scales;
  return from_cuda(mxk::launch_gemm_mx(A->fmt, B->fmt, A->data, A->scales, B->data, B->scales,
                                       C->data, MX_DT_F32, N, M, N, K, nullptr, 0, e,
                                       static_cast<cudaStream_t>(stream)));
}

mx_status gemm_dequant_splitk(const void* A, int32_t a_dtype, int64_t M, int64_t lda,
                              const mx_tensor* B, const mx_epilogue* epi, void* C,
                              int32_t c_dtype, int64_t ldc, void* workspace,
                              size_t workspace_bytes, void* stream) {
  mx_status s;
  if (a_dtype != MX_DT_F16 && a_dtype != MX_DT_BF16) return MX_ERR_INVALID_ARG;
  if (c_dtype != MX_DT_F32 && c_dtype != MX_DT_BF16) return MX_ERR_INVALID_ARG;
  if ((s = check_tensor(B)) != MX_OK) return s;
  mxk::Epilogue e;
  if ((s = epilogue_from(epi, &e)) != MX_OK) return s;
  if (M < 0 || M > kMaxDim) return MX_ERR_SHAPE;
  const int64_t N = B->outer, K = B->K;
  if (M == 0 || N == 0) return MX_OK;
  if (K == 0 || K % 64) return MX_ERR_SHAPE;
  if (!A || !C) return MX_ERR_INVALID_ARG;
  if (lda < K || lda % 8) return MX_ERR_SHAPE;
  const int64_t eb = (c_dtype == MX_DT_BF16) ? 2 : 4;
  if (ldc < N || (ldc * eb) % 16) return MX_ERR_SHAPE;
  if (!aligned16(A) || !aligned16(C) || (workspace && !aligned16(workspace)))
    return MX_ERR_ALIGN;
  if ((s = check_device()) != MX_OK) return s;
  return from_cuda(mxk::launch_gemm_dequant(a_dtype, A, lda, B->fmt, B->data, B->scales, C,
                                            c_dtype, ldc, M, N, K, e, workspace,
                                            workspace_bytes,
                                            static_cast<cudaStream_t>(stream)));
}

mx_status gemm_dequant(const void* A, int32_t a_dtype, int64_t M, int64_t lda,
                       const mx_tensor* B, const mx_epilogue* epi, void* C, int32_t c_dtype,
                       int64_t ldc, void* stream) {
  return gemm_dequant_splitk(A, a_dtype, M, lda, B, epi, C, c_dtype, ldc, nullptr, 0, stream);
}

size_t gemm_dequant_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || K % 64 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
    return 0;
  if (check_device() != MX_OK) return 0;
  return mxk::dequant_workspace_bytes(M, N, K);
}

namespace {

mx_status attention(const void* Q, const void* K, const void* V, void* O, int32_t dtype,
                    int32_t o_dtype, int64_t BH, int64_t Lq, int64_t Lk, int64_t d, float scale,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype != MX_DT_F16 && dtype != MX_DT_BF16) return MX_ERR_INVALID_ARG;
  if (o_dtype != MX_DT_F32 && o_dtype != MX_DT_BF16 && o_dtype != MX_DT_F16)
    return MX_ERR_INVALID_ARG;
  if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f) return MX_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return MX_ERR_SHAPE;
  if (BH < 0 || Lq < 0 || Lk < 0 || BH > 65535 || Lq > kMaxDim || Lk > kMaxDim)
    return MX_ERR_SHAPE;
  if (BH == 0 || Lq == 0) return MX_OK;
  if (Lk == 0) return MX_ERR_SHAPE;
  if (!Q || !K || !V || !O) return MX_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return MX_ERR_ALIGN;
  mx_status s = check_device();
  if (s != MX_OK) return s;
  if (workspace && !aligned16(workspace)) return MX_ERR_ALIGN;
  return from_cuda(mxk::launch_attention(dtype, Q, K, V, O, o_dtype, BH, Lq, Lk, d, scale,
                                         workspace, workspace_bytes,
                                         static_cast<cudaStream_t>(stream)));
}

}  // namespace

mx_status flash_attention(const void* Q, const void* K, const void* V, void* O, int32_t dtype,
                          int32_t o_dtype, int64_t BH, int64_t Lq, int64_t Lk, int64_t d,
                          float scale, void* stream) {
  return attention(Q, K, V, O, dtype, o_dtype, BH, Lq, Lk, d, scale, nullptr, 0, stream);
}

size_t flash_attention_workspace_bytes(int64_t BH, int64_t Lq, int64_t Lk, int64_t d) {
  if (BH <= 0 || Lq <= 0 || Lk <= 0 || BH > 65535 || Lq > kMaxDim || Lk > kMaxDim) return 0;
  if (d != 64 && d != 128) return 0;
  if (check_device() != MX_OK) return 0;
  return mxk::attention_workspace_bytes(BH, Lq, Lk, d);
}

mx_status flash_attention_splitkv(const void* Q, const void* K, const void* V, void* O,
                                  int32_t dtype, int32_t o_dtype, int64_t BH, int64_t Lq,
                                  int64_t Lk, int64_t d, float scale, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return attention(Q, K, V, O, dtype, o_dtype, BH, Lq, Lk, d, scale, workspace, workspace_bytes,
                   stream);
}

namespace {

bool is_page(int32_t page) { return page == 16 || page == 32 || page == 64 || page == 128; }

mx_status check_cache(const mx_kv_cache* c, mxk::KvCache* out) {
  if (!c) return MX_ERR_INVALID_ARG;
  if (c->fmt != MX_FMT_E4M3 && c->fmt != MX_FMT_E5M2 && c->fmt != MX_FMT_INT8)
    return MX_ERR_INVALID_ARG;
  if (!is_page(c->page) || (c->d != 64 && c->d != 128)) return MX_ERR_SHAPE;
  if (c->heads < 1 || c->heads > 65535 || c->pages < 1 ||
      c->pages > kMaxDim / (c->heads * c->page))
    return MX_ERR_SHAPE;
  if (!c->k_data || !c->v_data || !c->k_scales || !c->v_scales) return MX_ERR_INVALID_ARG;
  if (!aligned16(c->k_data) || !aligned16(c->v_data)) return MX_ERR_ALIGN;
  out->k = static_cast<uint8_t*>(c->k_data);
  out->v = static_cast<uint8_t*>(c->v_data);
  out->k_scales = c->k_scales;
  out->v_scales = c->v_scales;
  out->fmt = c->fmt;
  out->page = c->page;
  out->pages = c->pages;
  out->heads = c->heads;
  out->d = c->d;
  return MX_OK;
}

// Token and head strides of a tokens x heads x d operand of 16- or 32-bit
// elements: multiples of 8, heads not overlapping (a stride is free where
// there is only one of its kind).
mx_status check_strides(int64_t tokens, int64_t heads, int64_t ts, int64_t hs, int64_t d) {
  if (ts % 8 || hs % 8) return MX_ERR_SHAPE;
  if (heads > 1 && hs < d) return MX_ERR_SHAPE;
  if (tokens > 1 && ts < d) return MX_ERR_SHAPE;
  return MX_OK;
}

mx_status check_pages_call(int64_t requests, int64_t stride, int64_t width, int64_t stack_size,
                           int32_t page) {
  if (!is_page(page)) return MX_ERR_SHAPE;
  if (requests < 0 || requests > 16384 || width < 1 || stride < width || stack_size < 0 ||
      width > kMaxDim || stride > kMaxDim || stack_size > kMaxDim)
    return MX_ERR_SHAPE;
  return MX_OK;
}

}  // namespace

mx_status mx_kv_extend(const int32_t* lens, const int32_t* new_tokens, int64_t requests,
                       int32_t* table, int64_t table_stride, int64_t table_width,
                       const int32_t* stack, int64_t stack_size, const int32_t* count,
                       int32_t page, int32_t* lens_out, int32_t* cu, int64_t* slots,
                       int64_t max_tokens, int32_t* counts_out, void* stream) {
  mx_status s = check_pages_call(requests, table_stride, table_width, stack_size, page);
  if (s != MX_OK) return s;
  if (max_tokens < 0 || max_tokens > kMaxDim) return MX_ERR_SHAPE;
  if (requests > 0 && (!lens || !new_tokens || !table || !lens_out)) return MX_ERR_INVALID_ARG;
  if ((stack_size > 0 && !stack) || (max_tokens > 0 && !slots) || !count || !cu || !counts_out)
    return MX_ERR_INVALID_ARG;
  if ((s = check_device()) != MX_OK) return s;
  return from_cuda(mxk::launch_kv_extend(lens, new_tokens, requests, table, table_stride,
                                         table_width, stack, stack_size, count, page, lens_out,
                                         cu, slots, max_tokens, counts_out,
                                         static_cast<cudaStream_t>(stream)));
}

mx_status mx_kv_truncate(const int32_t* lens, const int32_t* keep, int64_t requests,
                         int32_t* table, int64_t table_stride, int64_t table_width,
                         int32_t* stack, int64_t stack_size, const int32_t* count, int32_t page,
                         int32_t* lens_out, int32_t* counts_out, void* stream) {
  mx_status s = check_pages_call(requests, table_stride, table_width, stack_size, page);
  if (s != MX_OK) return s;
  if (requests > 0 && (!lens || !keep || !table || !lens_out)) return MX_ERR_INVALID_ARG;
  if ((stack_size > 0 && !stack) || !count || !counts_out) return MX_ERR_INVALID_ARG;
  if ((s = check_device()) != MX_OK) return s;
  return from_cuda(mxk::launch_kv_truncate(lens, keep, requests, table, table_stride,
                                           table_width, stack, stack_size, count, page, lens_out,
                                           counts_out, static_cast<cudaStream_t>(stream)));
}

mx_status mx_kv_append(const mx_kv_cache* cache, const void* K, const void* V, int32_t dtype,
                       int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                       int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                       void* stream) {
  mxk::KvCache c;
  mx_status s = check_cache(cache, &c);
  if (s != MX_OK) return s;
  if (dtype != MX_DT_F16 && dtype != MX_DT_BF16) return MX_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > kMaxDim) return MX_ERR_SHAPE;
  if (tokens == 0) return MX_OK;
  if (!K || !V || !slots) return MX_ERR_INVALID_ARG;
  if ((s = check_strides(tokens, c.heads, k_token_stride, k_head_stride, c.d)) != MX_OK) return s;
  if ((s = check_strides(tokens, c.heads, v_token_stride, v_head_stride, c.d)) != MX_OK) return s;
  if (!aligned16(K) || !aligned16(V)) return MX_ERR_ALIGN;
  if ((s = check_device()) != MX_OK) return s;
  return from_cuda(mxk::launch_kv_append(c, K, V, dtype, tokens, k_token_stride, k_head_stride,
                                         v_token_stride, v_head_stride, slots,
                                         static_cast<cudaStream_t>(stream)));
}

size_t mx_kv_attention_workspace_bytes(int64_t q_heads, int64_t heads, int64_t d, int64_t max_q) {
  if (heads < 1 || heads > 65535 || q_heads < 1 || q_heads % heads || (d != 64 && d != 128) ||
      max_q < 1 || max_q > kMaxDim)
    return 0;
  if (check_device() != MX_OK) return 0;
  return mxk::kv_attention_workspace_bytes(q_heads, heads, d, max_q);
}

mx_status mx_kv_attention(const void* Q, int32_t dtype, int64_t tokens, int64_t q_heads,
                          int64_t q_token_stride, int64_t q_head_stride,
                          const mx_kv_cache* cache, const int32_t* table, int64_t table_stride,
                          int64_t table_width, const int32_t* lens, const int32_t* cu,
                          int64_t requests, int64_t max_q, void* O, int32_t o_dtype,
                          int64_t o_token_stride, int64_t o_head_stride, int32_t causal,
                          int64_t window, float scale, void* workspace, size_t workspace_bytes,
                          void* stream) {
  mxk::KvAttn a{};
  mx_status s = check_cache(cache, &a.cache);
  if (s != MX_OK) return s;
  if (dtype != MX_DT_F16 && dtype != MX_DT_BF16) return MX_ERR_INVALID_ARG;
  if (o_dtype != MX_DT_F32 && o_dtype != MX_DT_BF16 && o_dtype != MX_DT_F16)
    return MX_ERR_INVALID_ARG;
  if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f) return MX_ERR_INVALID_ARG;
  if ((causal != 0 && causal != 1) || window < 0) return MX_ERR_INVALID_ARG;
  const int64_t d = a.cache.d;
  if (q_heads < 1 || q_heads % a.cache.heads) return MX_ERR_SHAPE;
  // rows of one cache head are counted in 32 bits, rounded up to whole tiles
  if (tokens < 0 || tokens > (kMaxDim - 1024) / (q_heads / a.cache.heads)) return MX_ERR_SHAPE;
  if (requests < 0 || requests > kMaxDim || max_q < 0 || max_q > kMaxDim) return MX_ERR_SHAPE;
  if (table_width < 1 || table_stride < table_width || table_width > kMaxDim ||
      table_stride > kMaxDim)
    return MX_ERR_SHAPE;
  if (tokens == 0 || requests == 0) return MX_OK;
  if (!Q || !O || !table || !lens || !cu) return MX_ERR_INVALID_ARG;
  if ((s = check_strides(tokens, q_heads, q_token_stride, q_head_stride, d)) != MX_OK) return s;
  if ((s = check_strides(tokens, q_heads, o_token_stride, o_head_stride, d)) != MX_OK) return s;
  if (!aligned16(Q) || !aligned16(O) || (workspace && !aligned16(workspace))) return MX_ERR_ALIGN;
  if ((s = check_device()) != MX_OK) return s;
  a.Q = Q;
  a.dtype = dtype;
  a.tokens = tokens;
  a.q_heads = q_heads;
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.table = table;
  a.table_stride = table_stride;
  a.width = table_width;
  a.lens = lens;
  a.cu = cu;
  a.requests = requests;
  a.max_q = max_q;
  a.O = O;
  a.o_dtype = o_dtype;
  a.o_ts = o_token_stride;
  a.o_hs = o_head_stride;
  a.causal = causal;
  a.window = window;
  a.scale = scale;
  a.ws = workspace;
  a.ws_bytes = workspace_bytes;
  return from_cuda(mxk::launch_kv_attention(a, static_cast<cudaStream_t>(stream)));
}

mx_status gemm_f16(const void* A, const void* B, float* C, int32_t ab_dtype, int64_t M,
                   int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc,
                   void* stream) {
  return f16_product(A, B, nullptr, C, ab_dtype, M, N, K, lda, ldb, ldc, nullptr, 0, stream);
}

size_t gemm_f16_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return 0;
  if (check_device() != MX_OK) return 0;
  return mxk::gemm_workspace_bytes(0, M, N, K);
}

mx_status gemm_f16_splitk(const void* A, const void* B, float* C, int32_t ab_dtype, int64_t M,
                          int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (workspace && !aligned16(workspace)) return MX_ERR_ALIGN;
  return f16_product(A, B, nullptr, C, ab_dtype, M, N, K, lda, ldb, ldc, workspace,
                     workspace_bytes, stream);
}

mx_status gemm_f16_fused(const void* A, const void* B, const mx_epilogue* epi, float* C,
                         int32_t ab_dtype, int64_t M, int64_t N, int64_t K, int64_t lda,
                         int64_t ldb, int64_t ldc, void* stream) {
  return f16_product(A, B, epi, C, ab_dtype, M, N, K, lda, ldb, ldc, nullptr, 0, stream);
}

mx_status mx_last_error(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return MX_ERR_CUDA;
  cudaError_t e1 = cudaSuccess, e2 = cudaSuccess;
  const unsigned a = mxk::fetch_and_clear_status_quantize(&e1);
  const unsigned b = mxk::fetch_and_clear_status_gemm(&e2);
  cudaError_t e3 = cudaSuccess, e4 = cudaSuccess;
  const unsigned c = mxk::fetch_and_clear_status_dq(&e3);
  const unsigned d = mxk::fetch_and_clear_status_attn(&e4);
  cudaError_t e5 = cudaSuccess, e6 = cudaSuccess, e7 = cudaSuccess;
  const unsigned f = mxk::fetch_and_clear_status_dqd(&e5);
  const unsigned g = mxk::fetch_and_clear_status_kv(&e6) | mxk::fetch_and_clear_status_kvp(&e7);
  if (e1 != cudaSuccess || e2 != cudaSuccess || e3 != cudaSuccess || e4 != cudaSuccess ||
      e5 != cudaSuccess || e6 != cudaSuccess || e7 != cudaSuccess)
    return MX_ERR_CUDA;
  if ((a | b | c | d | f | g) & mxk::STATUS_TIMEOUT) return MX_ERR_TIMEOUT;
  return MX_OK;
}

mx_status mx_selftest_wait_timeout(int64_t limit_cycles, void* stream) {
  if (limit_cycles < 1 || limit_cycles > (int64_t{1} << 40)) return MX_ERR_INVALID_ARG;
  mx_status s = check_device();
  if (s != MX_OK) return s;
  return from_cuda(
      mxk::launch_selftest_timeout(limit_cycles, static_cast<cudaStream_t>(stream)));
}

mx_status mx_scales_to_rowmajor(const uint8_t* tiled, uint8_t* rowmajor, int64_t outer,
                                int64_t K) {
  if (outer < 0 || K < 0 || K % 32) return MX_ERR_SHAPE;
  if ((outer > 0 && K > 0) && (!tiled || !rowmajor)) return MX_ERR_INVALID_ARG;
  const int64_t nb = K / 32, ka = mxk::sf_k_atoms(K);
  for (int64_t r = 0; r < outer; ++r)
    for (int64_t j = 0; j < nb; ++j) rowmajor[r * nb + j] = tiled[mxk::sf_offset(r, j, ka)];
  return MX_OK;
}

const char* mx_status_string(int32_t status) {
  switch (status) {
    case MX_OK: return "MX_OK";
    case MX_ERR_INVALID_ARG: return "MX_ERR_INVALID_ARG";
    case MX_ERR_SHAPE: return "MX_ERR_SHAPE";
    case MX_ERR_ALIGN: return "MX_ERR_ALIGN";
    case MX_ERR_UNSUPPORTED: return "MX_ERR_UNSUPPORTED";
    case MX_ERR_CUDA: return "MX_ERR_CUDA";
    case MX_ERR_TIMEOUT: return "MX_ERR_TIMEOUT";
    default: return "MX_ERR_UNKNOWN";
  }
}

int32_t mx_version(void) { return 200; }

mx_status mx_set_tile_width(int32_t tbn) {
  if (tbn != 0 && tbn != 128 && tbn != 256) return MX_ERR_INVALID_ARG;
  mxk::gemm_force_tile_width(tbn);
  return MX_OK;
}

}  // extern "C"
#pragma GCC visibility pop
