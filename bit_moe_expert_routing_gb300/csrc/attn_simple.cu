// Attention over the 4-bit cache on the CUDA cores.
//
// One CTA per (step token, kv head, eight of its query heads), a warp per
// query head. Keys and values are dequantised 32 positions at a time into
// shared memory; lane l scores key l, and holds the output dimensions l, l +
// 32, ... The running maximum and sum of the softmax make it one pass.
#include "kv.cuh"

namespace moe {
namespace {

constexpr int kKeys = 32, kHeads = 8;

template <int DIM>
__global__ void __launch_bounds__(kHeads * 32) attention_simple_kernel(const AttnArgs a, int max_rows) {
  __shared__ float q[kHeads][DIM];
  __shared__ float t[kKeys][DIM + 1];
  const int i = blockIdx.x, kvh = blockIdx.y, hs = blockIdx.z * kHeads;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int b = kv_seq_of(a.kv, i);
  const SeqInfo si = kv_seq(a.kv, b);
  if (si.n_new * a.group <= max_rows) return;
  const int pos = si.kv - (si.first + si.n_new - i);
  const bool mine = hs + warp < a.group;
  const int head = kvh * a.group + hs + warp;
  if (mine)
    for (int d = lane; d < DIM; d += 32) q[warp][d] = bf16_to_f32(a.q[i * a.q_stride + head * DIM + d]);
  float m = -INFINITY, l = 0.f, o[DIM / 32];
#pragma unroll
  for (int j = 0; j < DIM / 32; ++j) o[j] = 0.f;
  const int lo = a.window ? max(0, pos + 1 - a.window) : 0;
  const int page = 1 << a.kv.page_bits;
  for (int k0 = 0; k0 <= pos; k0 += kKeys) {
    if (k0 + kKeys <= lo && k0 >= a.sinks) {
      k0 = lo / kKeys * kKeys - kKeys;
      continue;
    }
    float p = 0.f, alpha = 1.f;
    bool seen = false;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
      for (int e = threadIdx.x; e < kKeys * (DIM / 8); e += kHeads * 32) {
        const int key = e / (DIM / 8), w = e % (DIM / 8), kp = k0 + key;
        uint32_t v[4] = {0, 0, 0, 0};
        long long row = -1;
        if (kp <= pos && (kp >= lo || kp < a.sinks)) row = kv_page_row(a.kv, b, kp >> a.kv.page_bits, kvh);
        if (row >= 0) {
          row += kp & (page - 1);
          const long long g = row * (DIM / 64) + w / 8;
          const __nv_bfloat16 s = __ushort_as_bfloat16(a.kv.scales[which][g]);
          const __nv_bfloat16 z = __ushort_as_bfloat16(a.kv.biases[which][g]);
          dq8_bf16(a.kv.codes[which][row * (DIM / 8) + w], __halves2bfloat162(s, s), __halves2bfloat162(z, z), v);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          t[key][w * 8 + 2 * c] = bf16lo(v[c]);
          t[key][w * 8 + 2 * c + 1] = bf16hi(v[c]);
        }
      }
      __syncthreads();
      if (which == 0) {
        const int kp = k0 + lane;
        seen = kp <= pos && (kp >= lo || kp < a.sinks);
        if (seen) {
          const int pg = kp >> a.kv.page_bits;
          const int e = pg < a.kv.table_stride ? a.kv.table[(long long)b * a.kv.table_stride + pg] : -1;
          seen = e >= 0 && e < a.kv.n_pages;
        }
        float s = 0.f;
        for (int d = 0; d < DIM; ++d) s += q[warp][d] * t[lane][d];
        s = seen ? s * a.scale : -INFINITY;
        float mx = s;
        for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, off));
        const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;
        alpha = __expf(m - ref);
        p = __expf(s - ref);
        float sum = p;
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(~0u, sum, off);
        l = l * alpha + sum;
        m = mn;
      } else {
#pragma unroll
        for (int j = 0; j < DIM / 32; ++j) {
          float acc = o[j] * alpha;
          for (int key = 0; key < kKeys; ++key) acc += __shfl_sync(~0u, p, key) * t[key][lane + 32 * j];
          o[j] = acc;
        }
      }
    }
  }
  if (!mine) return;
  const long long at = (long long)i * a.heads + head;
#pragma unroll
  for (int j = 0; j < DIM / 32; ++j) a.out[at * DIM + lane + 32 * j] = f32_to_bf16(l != 0.f ? o[j] / l : 0.f);
  if (a.lse && lane == 0) a.lse[at] = l != 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t attention_simple(const AttnArgs& a, int max_rows, const KvCall& c) {
  const dim3 grid(a.kv.n_tokens, a.kv.kv_heads, (a.group + kHeads - 1) / kHeads);
  if (a.kv.dim == 64)
    attention_simple_kernel<64><<<grid, kHeads * 32, 0, c.stream>>>(a, max_rows);
  else if (a.kv.dim == 128)
    attention_simple_kernel<128><<<grid, kHeads * 32, 0, c.stream>>>(a, max_rows);
  else
    attention_simple_kernel<256><<<grid, kHeads * 32, 0, c.stream>>>(a, max_rows);
  return c.launched("attention_simple");
}

}  // namespace moe
