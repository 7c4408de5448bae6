// C entry points of the 4-bit key/value cache and its attention.
#include "kv_host.cuh"

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
  return status_of(attend(g, few, workspace, begin_call(stream, opt)));
}

}  // extern "C"
