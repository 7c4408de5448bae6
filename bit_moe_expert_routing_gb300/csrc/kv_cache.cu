// The 4-bit key/value cache: quantising a step's tokens into their pages, and
// reading tokens back.
//
// Per group of 64 elements of a head: bias b = min, scale s = bf16((max -
// min) / 15), code q = clamp(rne((x - b) / s), 0, 15); the stored value is
// bf16(s q + b). Both kernels move 2.5625 bytes per element and do a few
// operations on each: memory sets their time.
#include "kv.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Page row of step token i for kv head h, or -1: padding, or no page.
__device__ __forceinline__ long long token_row(const KvArgs& a, int i, int h) {
  const int b = kv_seq_of(a, i);
  const int pos = a.kv_len[b] - (a.q_off[b + 1] - i);
  if (pos < 0) return -1;
  if (pos >= a.max_kv) {
    report(a.hdr, MOE_ERR_DEVICE_CHECK, kKvBadBatch);
    return -1;
  }
  const long long r = kv_page_row(a, b, pos >> a.page_bits, h);
  return r < 0 ? r : r + (pos & ((1 << a.page_bits) - 1));
}

// One thread per 8 elements (one code word), 8 neighbouring lanes per group.
// blockIdx.y: 0 keys, 1 values.
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvArgs a, const uint16_t* k, long long ks,
                                                             const uint16_t* v, long long vs) {
  const int which = blockIdx.y;
  const int words = a.dim / 8;  // per head row: 8, 16 or 32
  const long long idx = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long row = idx / words;
  const int w = int(idx % words);
  if (row >= (long long)a.n_tokens * a.kv_heads) return;  // whole groups of 8 lanes leave together
  const int i = int(row / a.kv_heads), h = int(row % a.kv_heads);
  const uint16_t* src = which ? v + i * vs : k + i * ks;
  const uint4 x4 = *reinterpret_cast<const uint4*>(src + h * a.dim + w * 8);
  const uint32_t xs[4] = {x4.x, x4.y, x4.z, x4.w};
  float x[8];
  bool bad = false;
  float lo = kKvLimit, hi = -kKvLimit;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float f = (j & 1) ? bf16hi(xs[j / 2]) : bf16lo(xs[j / 2]);
    if (!(fabsf(f) <= kKvLimit)) {
      bad = true;
      f = f != f ? 0.f : copysignf(kKvLimit, f);
    }
    x[j] = f;
    lo = fminf(lo, f);
    hi = fmaxf(hi, f);
  }
  const unsigned lanes = 0xffu << (threadIdx.x & 24);  // this group's eight lanes
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(lanes, lo, off));
    hi = fmaxf(hi, __shfl_xor_sync(lanes, hi, off));
  }
  if (lo == 0.f) lo = 0.f;  // one zero: a minimum of -0 and +0 may be either
  const uint16_t sb = f32_to_bf16(__fdiv_rn(hi - lo, 15.f));
  const float s = bf16_to_f32(sb);
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = s > 0.f ? fminf(rintf(__fdiv_rn(x[j] - lo, s)), 15.f) : 0.f;  // x >= lo
    word |= uint32_t(q) << (4 * j);
  }
  const long long dst = token_row(a, i, h);
  if (dst < 0) return;
  if (bad) report(a.hdr, MOE_ERR_DEVICE_CHECK, kKvBadNumber);
  a.codes[which][dst * words + w] = word;
  if ((w & 7) == 0) {
    a.scales[which][dst * (a.dim / 64) + w / 8] = sb;
    a.biases[which][dst * (a.dim / 64) + w / 8] = f32_to_bf16(lo);
  }
}

// One thread per code word.
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvArgs a, uint16_t* k, uint16_t* v) {
  const int which = blockIdx.y;
  uint16_t* out = which ? v : k;
  if (!out) return;
  const int words = a.dim / 8;
  const long long idx = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long row = idx / words;
  const int w = int(idx % words);
  if (row >= (long long)a.n_tokens * a.kv_heads) return;
  const int i = int(row / a.kv_heads), h = int(row % a.kv_heads);
  const long long src = token_row(a, i, h);
  uint32_t o[4] = {0, 0, 0, 0};
  if (src >= 0) {
    const long long g = src * (a.dim / 64) + w / 8;
    const __nv_bfloat16 s = __ushort_as_bfloat16(a.scales[which][g]), b = __ushort_as_bfloat16(a.biases[which][g]);
    dq8_bf16(a.codes[which][src * words + w], __halves2bfloat162(s, s), __halves2bfloat162(b, b), o);
  }
  *reinterpret_cast<uint4*>(out + row * a.dim + w * 8) = make_uint4(o[0], o[1], o[2], o[3]);
}

dim3 grid_of(const KvArgs& a) {
  const long long n = (long long)a.n_tokens * a.kv_heads * (a.dim / 8);
  return dim3(unsigned((n + kThreads - 1) / kThreads), 2);
}

}  // namespace

cudaError_t kv_append(const KvArgs& a, const uint16_t* k, long long ks, const uint16_t* v, long long vs,
                      const KvCall& c) {
  kv_append_kernel<<<grid_of(a), kThreads, 0, c.stream>>>(a, k, ks, v, vs);
  return c.launched("kv_append");
}

cudaError_t kv_read(const KvArgs& a, uint16_t* k, uint16_t* v, const KvCall& c) {
  kv_read_kernel<<<grid_of(a), kThreads, 0, c.stream>>>(a, k, v);
  return c.launched("kv_read");
}

}  // namespace moe
