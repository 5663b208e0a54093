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

// Pages that several requests hold (kvshare.cu): refs counts a page's holders
// beyond the first.
struct KvShare {
  const int* lens;
  const int* change;          // release: tokens kept; fork: tokens shared; own: new tokens
  int64_t requests;
  const int* src;             // fork
  const int* dst;
  int64_t forks;
  int* table;
  int64_t table_stride, width;
  int* stack;
  int64_t stack_size;
  const int* count;
  int* refs;
  int64_t pages;
  int page;
  int* lens_out;              // own: the new tokens that are allowed
  int* copies;                // own: requests x (from, to, tokens)
  int* counts_out;
};
cudaError_t launch_kv_release(const KvShare& q, cudaStream_t st);
cudaError_t launch_kv_fork(const KvShare& q, cudaStream_t st);
cudaError_t launch_kv_own(const KvCache& c, const KvShare& q, cudaStream_t st);

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

// Shared prefixes (kvshared.cu).  The attention kernels' SH variants take a list of
// entries instead of requests: the rows of a group over its prefix, or a request's rows
// over its keys behind the prefix.  Each row that has both leaves its state -- O before the
// division, the reference m and the sum l -- of either in memory, a row for each (token, query
// head): whole where a unit is not cut, or in the parts of the workspace; rec says where.
struct KvEntry {
  int q0, q1;                  // rows of Q
  int len;                     // keys up to here
  int start;                   // the first key
  int row;                     // of the table
  int prefix;                  // the rows of a group: all of them see all of the keys
  float prefix_time, own_time; // of a group, in SM-microseconds: for how many SMs each pass gets
};
// rec of a row: {its first part's slot, the CTA that has it, the parts (0: the state is
// whole), the row in the unit and flags}.  Part i > 0 stands in slot 2 (CTA + i).
constexpr int KV_REC_PREFIX = 1 << 16;      // the row has a prefix's state besides
constexpr int KV_REC_DONE = 1 << 17;        // the row is written
struct KvStates {
  float* o;                    // rows x d
  float2* ml;                  // rows: m, l
  int4* rec;                   // rows
};
struct KvPassArgs {
  const KvEntry* list;
  int64_t entries;
  KvStates prefix, own;
  const KvEntry* groups;       // two passes beside one another: whose times share the SMs out
  int n_groups;                // (0: each pass takes what it finds)
};
constexpr int KV_SPLIT_GROUPS = 512;        // at the most: a lane reads 16
// Which kernel a pass takes: rows of a unit 8 or 16 (kvattn.cu) or 256 (kvprompt.cu),
// for entries of so many rows a cache head.
int kv_pass_unit(int64_t rows);
int kv_pass_ctas(int unit, int64_t d, int sms);
size_t kv_pass_workspace_bytes(int unit, int64_t d, int sms);
int kv_sm_count();
// Launched as a programmatic dependent; `wait`: what it reads was written by the kernel
// before it.  KvAttn: Q, cache, table and O, and the pass's workspace.
cudaError_t launch_kv_pass(const KvAttn& a, const KvPassArgs& pass, int unit, bool wait, int sms,
                           cudaStream_t st);

// The call: requests groups[g] .. groups[g + 1] - 1 share their first shared[g] tokens.
struct KvGroups {
  const int* groups;
  const int* shared;
  int64_t n;
};
size_t kv_attention_shared_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d,
                                           int64_t max_q, int64_t requests, int64_t groups);
cudaError_t launch_kv_attention_shared(const KvAttn& a, const KvGroups& g, cudaStream_t st);
void kv_set_shared_bytes(int64_t bytes);    // negative: the default

// Its kernel for many rows per request (kvprompt.cu), up to
// kv_prompt_max_requests() requests.
int64_t kv_prompt_max_requests();
size_t kv_prompt_workspace_bytes(int64_t d, int sms);
cudaError_t launch_kv_prompt(const KvAttn& a, int sms, const KvPassArgs* pass, bool wait, cudaStream_t st);
unsigned fetch_and_clear_status_kvp(cudaError_t* err);

}  // namespace mxk
