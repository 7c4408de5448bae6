// The 4-bit key/value cache: quantising a step's tokens into their pages, and
// reading tokens back.
//
// Per group of 64 elements of a head: bias b = min, scale s = bf16((max -
// min) / 15), code q = clamp(rne((x - b) / s), 0, 15); the stored value is
// bf16(s q + b). Both kernels move 2.5625 bytes per element: memory is the
// floor, and what they have to keep small beside it is the instructions per
// element and the chain of dependent loads in front of the data (token ->
// sequence -> length -> page). So a CTA takes a run of step tokens for one kv
// head, looks their slots up once, and every thread has all its data loads in
// flight together.
#include "kv.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Step tokens of a CTA: eight code words per thread when it is full.
template <int DIM>
constexpr int kRun = 8 * kThreads / (DIM / 8);

// Cache rows (for kv head `h`) of step tokens i0 .. i0 + n - 1, or -1:
// padding, or no page. One thread per token.
__device__ __forceinline__ void token_rows(const KvArgs& a, int i0, int n, int h, long long* rows) {
  for (int t = threadIdx.x; t < n; t += kThreads) {
    const int i = i0 + t, b = kv_seq_of(a, i);
    const int pos = a.kv_len[b] - (a.q_off[b + 1] - i);
    long long r = -1;
    if (pos >= a.max_kv) {
      report(a.hdr, MOE_ERR_DEVICE_CHECK, kKvBadBatch);
    } else if (pos >= 0) {
      r = kv_page_row(a, b, pos >> a.page_bits, h);
      if (r >= 0) r += pos & ((1 << a.page_bits) - 1);
    }
    rows[t] = r;
  }
  __syncthreads();
}

__device__ __forceinline__ __nv_bfloat162 pair(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t*>(&v); }

// (min x, -max x) of the group that eight neighbouring lanes hold; a NaN among them gives NaN.
__device__ __forceinline__ uint32_t group_range(const uint32_t (&x)[4], unsigned lanes) {
  const uint32_t lo = bits(__hmin2_nan(__hmin2_nan(pair(x[0]), pair(x[1])), __hmin2_nan(pair(x[2]), pair(x[3]))));
  const uint32_t hi = bits(__hmax2_nan(__hmax2_nan(pair(x[0]), pair(x[1])), __hmax2_nan(pair(x[2]), pair(x[3]))));
  const uint32_t neg = hi ^ 0x80008000u;
  __nv_bfloat162 m = __hmin2_nan(pair(__byte_perm(lo, neg, 0x5410)), pair(__byte_perm(lo, neg, 0x7632)));
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) m = __hmin2_nan(m, pair(__shfl_xor_sync(lanes, bits(m), off)));
  return bits(m);
}

// Eight elements as numbers of the cache's range: the nearest, NaN 0.
__device__ __noinline__ uint4 saturate8(uint4 x4) {
  uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int at = 16 * (j & 1);
    uint32_t e = (x[j / 2] >> at) & 0xFFFFu;
    if ((e & 0x7FFFu) > 0x7F80u)
      e = 0;
    else if ((e & 0x7FFFu) > 0x4780u)  // 2^16
      e = (e & 0x8000u) | 0x4780u;
    x[j / 2] = (x[j / 2] & ~(0xFFFFu << at)) | e << at;
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// Eight elements of a group (eight neighbouring lanes hold a group): their
// code word, and the group's scale and bias. `bad` is set if an element of
// the group is not a number of the cache's range.
__device__ __forceinline__ uint32_t quantise8(uint4 x4, uint16_t* scale, uint16_t* bias, bool* bad) {
  const unsigned lanes = 0xffu << (threadIdx.x & 24);
  uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
  uint32_t m = group_range(x, lanes);
  if (!(fmaxf(fabsf(bf16lo(m)), fabsf(bf16hi(m))) <= kKvLimit) || bf16lo(m) != bf16lo(m) || bf16hi(m) != bf16hi(m)) {
    *bad = true;  // (the eight lanes agree)
    const uint4 y = saturate8(x4);
    x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
    m = group_range(x, lanes);
  }
  const float lo = bf16lo(m) + 0.f;  // (one zero: a minimum of -0 and +0 may be either)
  const uint16_t sb = f32_to_bf16(__fdiv_rn(-bf16hi(m) - lo, 15.f));
  *scale = sb;
  *bias = f32_to_bf16(lo);
  const float s = bf16_to_f32(sb);
  float a[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) a[j] = ((j & 1) ? bf16hi(x[j / 2]) : bf16lo(x[j / 2])) - lo;
  if (s < 1e-30f) {  // 1 / s would overflow
    uint32_t word = 0;
    if (s > 0.f)
      for (int j = 0; j < 8; ++j) word |= uint32_t(fminf(rintf(__fdiv_rn(a[j], s)), 15.f)) << (4 * j);
    return word;
  }
  // q = rne(a / s) from a * (1 / s), which is at most one off, and only where
  // a / s is within a few ulp of a half: the remainder r = a - q s is exact in
  // fp32 (q s has 12 bits), and |r| >= s / 2 finds those and the ties. Adding
  // 1.5 * 2^23 rounds to the nearest integer and leaves it in the low bits. (a
  // / s is below 15.5, the scale being rounded by 2^-9 at most, so no code
  // passes 15 but in the subnormal range, left to the division above.)
  const float inv = __fdividef(1.f, s), half = 0.5f * s;
  constexpr float kMagic = 12582912.f;
  float r[8], worst = 0.f;
  uint32_t q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float g = __fmaf_rn(a[j], inv, kMagic);
    q[j] = __float_as_uint(g);
    r[j] = __fmaf_rn(kMagic - g, s, a[j]);
    worst = fmaxf(worst, fabsf(r[j]));
  }
  if (worst >= half) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = fabsf(r[j]);
      if (d > half || (d == half && (q[j] & 1u))) q[j] += r[j] > 0.f ? 1u : ~0u;
    }
  }
  // sum of q 16^j; the constant's bits in every q add up to a known multiple
  uint32_t word = 0;
#pragma unroll
  for (int j = 7; j >= 0; --j) word = word * 16u + q[j];
  return word - 0x4B400000u * 0x11111111u;
}

// CTA (run of step tokens, kv head, 0 keys / 1 values).
template <int DIM>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvArgs a, const uint16_t* k, long long ks,
                                                             const uint16_t* v, long long vs) {
  constexpr int W = DIM / 8, kPass = kThreads / W;  // code words of a head; tokens of one pass over the threads
  __shared__ long long rows[kRun<DIM>];
  const int h = blockIdx.y, which = blockIdx.z;
  const int i0 = blockIdx.x * kRun<DIM>, n = min(kRun<DIM>, a.n_tokens - i0);
  const int w = threadIdx.x % W, t0 = threadIdx.x / W;
  const long long stride = which ? vs : ks;
  const uint16_t* src = (which ? v : k) + i0 * stride + h * DIM + w * 8;
  uint32_t* codes = which ? a.codes[1] : a.codes[0];
  uint16_t* scales = which ? a.scales[1] : a.scales[0];
  uint16_t* biases = which ? a.biases[1] : a.biases[0];
  uint4 x[4];
  auto load = [&](int p) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + (p + j) * kPass;
      x[j] = t < n ? *reinterpret_cast<const uint4*>(src + t * stride) : make_uint4(0, 0, 0, 0);
    }
  };
  load(0);  // before the slots are looked up
  token_rows(a, i0, n, h, rows);
  bool bad = false;
#pragma unroll 1
  for (int p = 0; p < 8; p += 4) {
    if (p) {
      if (p * kPass >= n) break;
      load(p);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + (p + j) * kPass;
      uint16_t s, b;
      bool off = false;
      const uint32_t word = quantise8(x[j], &s, &b, &off);
      const long long row = t < n ? rows[t] : -1;
      if (row < 0) continue;
      bad |= off;
      codes[row * W + w] = word;
      if ((w & 7) == 0) {
        scales[row * (DIM / 64) + w / 8] = s;
        biases[row * (DIM / 64) + w / 8] = b;
      }
    }
  }
  if (bad) report(a.hdr, MOE_ERR_DEVICE_CHECK, kKvBadNumber);
}

template <int DIM>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvArgs a, uint16_t* k, uint16_t* v) {
  constexpr int W = DIM / 8, kPass = kThreads / W;
  __shared__ long long rows[kRun<DIM>];
  const int h = blockIdx.y, which = blockIdx.z;
  uint16_t* out = which ? v : k;
  if (!out) return;
  const int i0 = blockIdx.x * kRun<DIM>, n = min(kRun<DIM>, a.n_tokens - i0);
  const int w = threadIdx.x % W, t0 = threadIdx.x / W;
  const uint32_t* codes = which ? a.codes[1] : a.codes[0];
  const uint16_t* scales = which ? a.scales[1] : a.scales[0];
  const uint16_t* biases = which ? a.biases[1] : a.biases[0];
  token_rows(a, i0, n, h, rows);
  uint32_t c[8];
  uint16_t s[8], b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int t = t0 + j * kPass;
    const long long row = t < n ? rows[t] : -1;
    c[j] = s[j] = b[j] = 0;
    if (row >= 0) {
      c[j] = codes[row * W + w];
      s[j] = scales[row * (DIM / 64) + w / 8];
      b[j] = biases[row * (DIM / 64) + w / 8];
    }
  }
  uint16_t* dst = out + ((long long)i0 * a.kv_heads + h) * DIM + w * 8;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int t = t0 + j * kPass;
    if (t >= n) break;
    uint32_t o[4];
    const __nv_bfloat16 sj = __ushort_as_bfloat16(s[j]), bj = __ushort_as_bfloat16(b[j]);
    dq8_bf16(c[j], __halves2bfloat162(sj, sj), __halves2bfloat162(bj, bj), o);
    *reinterpret_cast<uint4*>(dst + (long long)t * a.kv_heads * DIM) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int DIM>
dim3 grid_of(const KvArgs& a) {
  return dim3(unsigned((a.n_tokens + kRun<DIM> - 1) / kRun<DIM>), unsigned(a.kv_heads), 2);
}

template <int DIM>
void launch_append(const KvArgs& a, const uint16_t* k, long long ks, const uint16_t* v, long long vs, cudaStream_t s) {
  kv_append_kernel<DIM><<<grid_of<DIM>(a), kThreads, 0, s>>>(a, k, ks, v, vs);
}
template <int DIM>
void launch_read(const KvArgs& a, uint16_t* k, uint16_t* v, cudaStream_t s) {
  kv_read_kernel<DIM><<<grid_of<DIM>(a), kThreads, 0, s>>>(a, k, v);
}

}  // namespace

cudaError_t kv_append(const KvArgs& a, const uint16_t* k, long long ks, const uint16_t* v, long long vs,
                      const KvCall& c) {
  (a.dim == 64 ? launch_append<64> : a.dim == 128 ? launch_append<128> : launch_append<256>)(a, k, ks, v, vs, c.stream);
  return c.launched("kv_append");
}

cudaError_t kv_read(const KvArgs& a, uint16_t* k, uint16_t* v, const KvCall& c) {
  (a.dim == 64 ? launch_read<64> : a.dim == 128 ? launch_read<128> : launch_read<256>)(a, k, v, c.stream);
  return c.launched("kv_read");
}

}  // namespace moe
