// kv_common.cuh -- the 8-bit paged key/value cache: one definition of its
// layout, shared by the kernels that write it (kvappend.cu) and read it
// (kvattn.cu, kvprompt.cu) and by the bookkeeping of its pages (kvpages.cu).
//
// A cache holds `pages` pages of P tokens (P = 16, 32, 64 or 128) for each of
// H heads of d values (64 or 128), keys and values apart.  A page of one head
// is P x d codes, contiguous (so that it is one TMA box), at
// ((page * H + head) * P + token) * d; its scale is one UE8M0 byte (value
// 2^(c - 127), 0xFF = NaN) at page * H + head.  Elements are E4M3, E5M2 or
// int8 codes; a value is code * scale.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace mxk {

struct KvCache {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_scales;
  uint8_t* v_scales;
  int fmt;
  int page;
  int64_t pages;
  int64_t heads;
  int64_t d;
};

__host__ __device__ __forceinline__ int kv_page_shift(int page) {
  return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
}

cudaError_t launch_kv_extend(const int* lens, const int* fresh, int64_t requests, int* table,
                             int64_t table_stride, int64_t width, const int* stack,
                             int64_t stack_size, const int* count, int page, int* lens_out,
                             int* cu, int64_t* slots, int64_t max_tokens, int* counts_out,
                             cudaStream_t st);
cudaError_t launch_kv_truncate(const int* lens, const int* keep, int64_t requests, int* table,
                               int64_t table_stride, int64_t width, int* stack,
                               int64_t stack_size, const int* count, int page, int* lens_out,
                               int* counts_out, cudaStream_t st);

// K and V: tokens x heads x d of dtype (DT_BF16 / DT_F16), strides in
// elements; slots: one per token.
cudaError_t launch_kv_append(const KvCache& c, const void* K, const void* V, int dtype,
                             int64_t tokens, int64_t k_ts, int64_t k_hs, int64_t v_ts,
                             int64_t v_hs, const int64_t* slots, cudaStream_t st);

// Attention of the queries of `requests` requests over the cache.
struct KvAttn {
  const void* Q;
  int dtype;
  int64_t tokens;             // rows of Q and O
  int64_t q_heads;
  int64_t q_ts, q_hs;         // strides of Q in elements: token, head
  KvCache cache;
  const int* table;
  int64_t table_stride, width;
  const int* lens;
  const int* cu;
  int64_t requests;
  int64_t max_q;
  void* O;
  int o_dtype;
  int64_t o_ts, o_hs;
  int causal;
  int64_t window;             // 0: none
  float scale;
  void* ws;
  size_t ws_bytes;
};
size_t kv_attention_workspace_bytes(int64_t q_heads, int64_t kv_heads, int64_t d, int64_t max_q);
cudaError_t launch_kv_attention(const KvAttn& a, cudaStream_t st);
unsigned fetch_and_clear_status_kv(cudaError_t* err);

// Its kernel for many rows per request (kvprompt.cu), up to
// kv_prompt_max_requests() requests.
int64_t kv_prompt_max_requests();
size_t kv_prompt_workspace_bytes(int64_t d, int sms);
cudaError_t launch_kv_prompt(const KvAttn& a, int sms, cudaStream_t st);
unsigned fetch_and_clear_status_kvp(cudaError_t* err);

}  // namespace mxk
