// Shared by the kernels of the 4-bit key/value cache and its attention.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr float kKvLimit = 65536.f;  // largest magnitude the cache holds

// Device view of moe_kv_cache and moe_kv_batch.
struct KvArgs {
  uint32_t* codes[2];  // keys, values
  uint16_t* scales[2];
  uint16_t* biases[2];
  WsHeader* hdr;
  const int32_t* q_off;
  const int32_t* kv_len;
  const int32_t* table;
  int table_stride;
  int n_seqs, n_tokens, max_new, max_kv;
  int n_pages, page_bits, kv_heads, dim;
};

// Device-side checks recorded in the cache's status word (its detail).
constexpr int kKvBadPage = 200, kKvBadNumber = 201, kKvBadBatch = 202;

// First page row (row = one head of one slot) of a sequence's page `j`, or -1
// (recorded) when the table has no valid entry for it.
__device__ __forceinline__ long long kv_page_row(const KvArgs& a, int seq, int j, int head) {
  int p = -1;
  if (j < a.table_stride) p = a.table[(long long)seq * a.table_stride + j];
  if (p < 0 || p >= a.n_pages) {
    report(a.hdr, MOE_ERR_DEVICE_CHECK, kKvBadPage);
    return -1;
  }
  return ((long long)p * a.kv_heads + head) << a.page_bits;
}

// Sequence of step token `i` (0 <= i < n_tokens): the last one whose first
// token is at or before it.
__device__ __forceinline__ int kv_seq_of(const KvArgs& a, int i) {
  int lo = 0, hi = a.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.q_off[mid] <= i)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

struct SeqInfo {
  int first, n_new, kv;  // first step token, step tokens, positions
};
// A sequence's sizes with the host's bounds applied (a sequence past them is
// recorded and cut, so that no index leaves its buffer).
__device__ __forceinline__ SeqInfo kv_seq(const KvArgs& a, int b) {
  SeqInfo s;
  s.first = a.q_off[b];
  s.n_new = a.q_off[b + 1] - s.first;
  s.kv = a.kv_len[b];
  if (s.first < 0 || s.n_new < 0 || s.n_new > a.max_new || s.first > a.n_tokens - s.n_new || s.kv < 0 ||
      s.kv > a.max_kv) {
    report(a.hdr, MOE_ERR_DEVICE_CHECK, kKvBadBatch);
    s.first = s.n_new = s.kv = 0;
  }
  return s;
}

// One call: its stream and its copy of the options. launched() counts a
// kernel (and times it when that is on) and returns the launch's error.
struct KvCall {
  Options opt;
  cudaStream_t stream;
  cudaError_t launched(const char* name) const {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) launch_done(opt, stream, name);
    return e;
  }
};

struct AttnArgs {
  KvArgs kv;
  const uint16_t* q;
  long long q_stride;
  uint16_t* out;
  float* lse;
  int heads, group;  // query heads, query heads per kv head
  int window, sinks;
  float scale;
};

cudaError_t kv_append(const KvArgs& a, const uint16_t* k, long long ks, const uint16_t* v, long long vs,
                      const KvCall& c);
cudaError_t kv_read(const KvArgs& a, uint16_t* k, uint16_t* v, const KvCall& c);
// Sequences with at most max_rows rows (step tokens x query heads per kv head).
size_t attention_few_workspace(const AttnArgs& a, int max_rows);
long long attention_few_items(const AttnArgs& a, int max_rows);  // (sequence, kv head, group of rows), at most
// `beside`: launched behind the many-row kernels of the same call, on other
// sequences and another part of the workspace, so it does not wait for them.
cudaError_t attention_few(const AttnArgs& a, int max_rows, void* ws, bool beside, const KvCall& c);
// Sequences with more rows than that.
size_t attention_many_workspace(const AttnArgs& a);
cudaError_t attention_many(const AttnArgs& a, int max_few, void* ws, const KvCall& c);

}  // namespace moe
