// C entry points of the 4-bit key/value cache and its attention: argument
// checks on the host and the choice of kernels.
#include <algorithm>
#include <cmath>

#include "kv.cuh"

namespace moe {
namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

moe_status make_args(const moe_kv_cache* c, const moe_kv_batch* b, KvArgs* a) {
  if (!c || !b) return MOE_ERR_ARG;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_ERR_SHAPE;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return MOE_ERR_SHAPE;
  if (c->kv_heads < 1 || c->kv_heads > 256 || c->n_pages < 1) return MOE_ERR_SHAPE;
  if (b->n_seqs < 0 || b->n_tokens < 0 || b->n_tokens > kMaxTokens || b->n_seqs > 65535) return MOE_ERR_ARG;
  if (b->max_new < 0 || b->max_kv < 0 || b->max_kv > (1 << 24) || b->table_stride < 0) return MOE_ERR_ARG;
  const void* arrays[] = {c->k_codes, c->k_scales, c->k_biases, c->v_codes, c->v_scales, c->v_biases};
  for (const void* p : arrays)
    if (!p || !aligned(p, 16)) return MOE_ERR_ARG;
  if (!c->status || !aligned(c->status, 256)) return MOE_ERR_ARG;
  if (b->n_tokens > 0) {
    if (b->n_seqs < 1 || b->max_new < 1 || !b->q_off || !b->kv_len || !b->block_table) return MOE_ERR_ARG;
    if (!aligned(b->q_off, 4) || !aligned(b->kv_len, 4) || !aligned(b->block_table, 4)) return MOE_ERR_ARG;
  }
  *a = KvArgs{{c->k_codes, c->v_codes},
              {c->k_scales, c->v_scales},
              {c->k_biases, c->v_biases},
              static_cast<WsHeader*>(c->status),
              b->q_off,
              b->kv_len,
              b->block_table,
              b->table_stride,
              b->n_seqs,
              b->n_tokens,
              b->max_new < b->n_tokens ? b->max_new : b->n_tokens,
              b->max_kv,
              c->n_pages,
              __builtin_ctz(c->page_size),
              c->kv_heads,
              c->head_dim};
  return MOE_OK;
}

// A strided [n_tokens, heads, head_dim] operand.
bool operand_ok(const void* p, long long stride, int heads, int dim) {
  return p && aligned(p, 16) && stride % 8 == 0 && stride >= (long long)heads * dim;
}

moe_status check_attention(const KvArgs& kv, const moe_attention* a) {
  if (!a) return MOE_ERR_ARG;
  if (a->heads < kv.kv_heads || a->heads % kv.kv_heads || a->heads / kv.kv_heads > 64) return MOE_ERR_SHAPE;
  if (a->window < 0 || a->sinks < 0 || !std::isfinite(a->scale)) return MOE_ERR_ARG;
  return MOE_OK;
}

// Sequences with at most this many rows (step tokens x query heads per kv
// head) take the few-row kernel. (One number for a call: the kernels ask it of
// every sequence.)
//
// The few-row kernel expands the codes again for every 32 rows (16 of 256
// dims); the many-row path expands them once, ahead, and then works in tiles
// of 256 rows (512 of 64 dims), mostly empty below that: measured, 8 query
// heads per kv head of 128 dims, 2 kv heads, one sequence of 64000 keys, 64
// rows 25 us few and 51 many, 128 rows 40 and 52, 256 rows 65 and 54; of 256
// dims, 64 rows 56 and 84, 128 rows 93 and 86. So 128 rows, 64 of 256 dims.
//
// With more rows the few-row kernel still wins as long as its items are at
// most two CTAs' worth per SM and their products few: the many-row path's
// launches and set-up take longer than the work. Few against many, us, 128
// dims: one sequence, 1024 rows over no context 9 and 14, over 1000 keys (2^28
// products) 17 and 21, over 8000 keys (2^31) 43 and 29; 8 sequences, 256 rows
// over 1000 keys (2^29) 19 and 22, over 8000 keys (2^32) 72 and 45. Over 360
// drawn sizes this choice is 1.1% slower than the better kernel on average and
// by more than 5% at 16 of them: many sequences of few keys on either side of
// the switch (46 sequences, 9 tokens over 41 keys, 48 heads over 8 of 256 dims,
// 64 us for 35; 17 sequences, 136 tokens over 312 keys, 8 heads over 8 of 64
// dims, 42 for 27).
int few_rows(const AttnArgs& a, const Options& o) {
  constexpr int kAny = 1 << 30;
  if (o.force_path) return o.force_path == 1 ? kAny : 0;
  long long keys = a.kv.max_kv;
  if (a.window > 0) keys = std::min(keys, (long long)a.window + a.sinks + a.kv.max_new);
  const double products = double(keys) * a.kv.n_tokens * a.heads * a.kv.dim * (a.kv.dim == 256 ? 2 : 1);
  if (products <= double(1 << 30) && attention_few_items(a, kAny) <= 2 * num_sms()) return kAny;
  return a.kv.dim == 256 ? 64 : 128;
}

bool any_many(const AttnArgs& a, int few) { return (long long)a.kv.max_new * a.group > few; }

// Whether a sequence may have so few; when the step's tokens are max_new for
// every sequence, all are alike.
bool any_few(const AttnArgs& a, int few) {
  return few > 0 && (!any_many(a, few) || (long long)a.kv.n_seqs * a.kv.max_new != a.kv.n_tokens);
}

// The few-row kernels' part of the workspace, before the many-row kernels'
// (both are used when a step has sequences of both kinds; always there, and as
// large whether items are cut or not, so that no smaller step needs more).
size_t few_bytes(const AttnArgs& a, int few) {
  return (attention_few_workspace(a, few) + 255) & ~size_t(255);
}

AttnArgs attn_args(const KvArgs& kv, const moe_attention* at) {
  AttnArgs g{};
  g.kv = kv;
  g.heads = at->heads;
  g.group = at->heads / kv.kv_heads;
  // A window that covers every position hides none: it is no window, and both numbers stay below 2^24, so that the
  // kernels' differences from positions (of padding, down to -2^20) stay within 32 bits.
  g.window = at->window < kv.max_kv ? at->window : 0;
  g.sinks = g.window ? std::min(at->sinks, kv.max_kv) : 0;
  g.scale = at->scale;
  return g;
}

moe_status status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

size_t workspace_bytes_for(const AttnArgs& a, int few) {
  return ((few_bytes(a, few) + (any_many(a, few) ? attention_many_workspace(a) : 0)) + 511) & ~size_t(255);
}

KvCall begin_call(void* stream, const Options& opt = options_snapshot()) {
  const KvCall c{opt, static_cast<cudaStream_t>(stream)};
  timing_begin(c.opt, c.stream);
  return c;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_kv_append(const moe_kv_cache* cache, const moe_kv_batch* batch, const uint16_t* k, long long k_stride,
                         const uint16_t* v, long long v_stride, void* stream) {
  KvArgs a;
  reset_launch_count();
  if (moe_status s = make_args(cache, batch, &a)) return s;
  if (a.n_tokens == 0) return MOE_OK;
  if (!operand_ok(k, k_stride, a.kv_heads, a.dim) || !operand_ok(v, v_stride, a.kv_heads, a.dim)) return MOE_ERR_ARG;
  return status_of(kv_append(a, k, k_stride, v, v_stride, begin_call(stream)));
}

moe_status moe_kv_read(const moe_kv_cache* cache, const moe_kv_batch* batch, uint16_t* k, uint16_t* v, void* stream) {
  KvArgs a;
  reset_launch_count();
  if (moe_status s = make_args(cache, batch, &a)) return s;
  if (!aligned(k, 16) || !aligned(v, 16)) return MOE_ERR_ARG;
  if (a.n_tokens == 0 || (!k && !v)) return MOE_OK;
  return status_of(kv_read(a, k, v, begin_call(stream)));
}

size_t moe_attention_workspace_size(const moe_kv_cache* cache, const moe_kv_batch* batch, const moe_attention* at) {
  KvArgs a;
  if (make_args(cache, batch, &a) || check_attention(a, at)) return 0;
  const AttnArgs g = attn_args(a, at);
  return workspace_bytes_for(g, few_rows(g, options_snapshot()));
}

moe_status moe_attention_forward(const moe_kv_cache* cache, const moe_kv_batch* batch, const moe_attention* at,
                                 const uint16_t* q, long long q_stride, uint16_t* out, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  KvArgs a;
  reset_launch_count();
  if (moe_status s = make_args(cache, batch, &a)) return s;
  if (moe_status s = check_attention(a, at)) return s;
  if (a.n_tokens == 0) return MOE_OK;
  if (!operand_ok(q, q_stride, at->heads, a.dim) || !out || !aligned(out, 16) || out == q) return MOE_ERR_ARG;
  if (lse && !aligned(lse, 4)) return MOE_ERR_ARG;
  // the options once: the kernels are those that the workspace was checked for, whatever other threads set meanwhile
  const Options opt = options_snapshot();
  AttnArgs g = attn_args(a, at);
  const int few = few_rows(g, opt);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < workspace_bytes_for(g, few)) return MOE_ERR_WORKSPACE;
  g.q = q;
  g.q_stride = q_stride;
  g.out = out;
  g.lse = lse;
  const KvCall c = begin_call(stream, opt);
  const bool many = any_many(g, few);
  if (many)
    if (cudaError_t e = attention_many(g, few, static_cast<char*>(workspace) + few_bytes(g, few), c)) return status_of(e);
  return any_few(g, few) ? status_of(attention_few(g, few, workspace, many, c)) : MOE_OK;
}

}  // extern "C"
