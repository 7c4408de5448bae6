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

// Step tokens of a CTA: eight code words per thread when it is full (append:
// four passes of sixteen elements).
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

// (min x, -max x) of the group that four neighbouring lanes hold, sixteen
// elements each; a NaN among them gives NaN.
__device__ __forceinline__ uint32_t group_range(const uint32_t (&x)[8], unsigned lanes) {
  __nv_bfloat162 lo = pair(x[0]), hi = lo;
#pragma unroll
  for (int j = 1; j < 8; ++j) lo = __hmin2_nan(lo, pair(x[j])), hi = __hmax2_nan(hi, pair(x[j]));
  const uint32_t neg = bits(hi) ^ 0x80008000u;
  __nv_bfloat162 m = __hmin2_nan(pair(__byte_perm(bits(lo), neg, 0x5410)), pair(__byte_perm(bits(lo), neg, 0x7632)));
#pragma unroll
  for (int off = 2; off >= 1; off >>= 1) m = __hmin2_nan(m, pair(__shfl_xor_sync(lanes, bits(m), off)));
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

struct Eight {  // elements minus the bias
  float2 a[4];
};

// Code word of eight elements, given as a = x - bias: rne(a / s), at most 15.
// inv: 1 / s, too large by 2^-21 to 2^-19 of it.
//
// q = rne(a * inv), found by adding 1.5 * 2^23, is one too large where a / s is
// a half or within 2^-15 below one, and right elsewhere. The remainder r = a -
// q s is exact in fp32 (q s has 12 bits), and r + s / 2 negative finds the
// latter, 0 the halves, of which odd q step down. As integers: bits(r + s / 2)
// < (q & 1). (Halves are common: bf16 elements lie on a grid. A branch for
// them is taken by most warps.) a / s is below 15.5, the scale being rounded by
// 2^-9 at most, so no code passes 15 but where the scale is subnormal, which
// is left to a division. Two elements per instruction where there is one.
__device__ __forceinline__ uint32_t codes8(const Eight& x, float s, float inv) {
  constexpr float kMagic = 12582912.f;
  const float2 magic = make_float2(kMagic, kMagic), minus = make_float2(-1.f, -1.f);
  const float half = 0.5f * s;
  uint32_t word = 0;
#pragma unroll
  for (int j = 3; j >= 0; --j) {
    const float2 g = __ffma2_rn(x.a[j], make_float2(inv, inv), magic);
    const float2 r = __ffma2_rn(__ffma2_rn(g, minus, magic), make_float2(s, s), x.a[j]);
    const float2 e = __fadd2_rn(r, make_float2(half, half));
#pragma unroll
    for (int i = 1; i >= 0; --i) {
      const uint32_t q = __float_as_uint(i ? g.y : g.x);
      // sum of q 16^j; the constant's bits in every q add up to a known multiple
      word = word * 16u + q;
      if (__float_as_int(i ? e.y : e.x) < int(q & 1u)) --word;
    }
  }
  return word - 0x4B400000u * 0x11111111u;
}
__device__ __noinline__ uint32_t codes8_by_division(Eight x, float s) {
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    word |= uint32_t(fminf(rintf(__fdiv_rn(j & 1 ? x.a[j / 2].y : x.a[j / 2].x, s)), 15.f)) << (4 * j);
  return word;
}

// Sixteen elements of a group (four neighbouring lanes hold a group): their
// code words, and the group's scale and bias. `bad` is set if an element of
// the group is not a number of the cache's range.
__device__ __forceinline__ uint2 quantise16(const uint4 (&x4)[2], uint16_t* scale, uint16_t* bias, bool* bad) {
  const unsigned lanes = 0xfu << (threadIdx.x & 28);
  uint32_t x[8] = {x4[0].x, x4[0].y, x4[0].z, x4[0].w, x4[1].x, x4[1].y, x4[1].z, x4[1].w};
  uint32_t m = group_range(x, lanes);
  if (!(fmaxf(fabsf(bf16lo(m)), fabsf(bf16hi(m))) <= kKvLimit) || bf16lo(m) != bf16lo(m) || bf16hi(m) != bf16hi(m)) {
    *bad = true;  // (the four lanes agree)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 y = saturate8(x4[i]);
      x[4 * i] = y.x, x[4 * i + 1] = y.y, x[4 * i + 2] = y.z, x[4 * i + 3] = y.w;
    }
    m = group_range(x, lanes);
  }
  const float lo = bf16lo(m) + 0.f;  // (one zero: a minimum of -0 and +0 may be either)
  const uint16_t sb = f32_to_bf16(__fdiv_rn(-bf16hi(m) - lo, 15.f));
  *scale = sb;
  *bias = f32_to_bf16(lo);
  const float s = bf16_to_f32(sb);
  const float inv = __fdividef(1.f, s) * (1.f + 0x1p-20f);
  uint32_t words[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    Eight a;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      a.a[j] = __fadd2_rn(make_float2(bf16lo(x[4 * i + j]), bf16hi(x[4 * i + j])), make_float2(-lo, -lo));
    words[i] = s >= 1e-30f ? codes8(a, s, inv) : s > 0.f ? codes8_by_division(a, s) : 0;  // (1 / s would overflow)
  }
  return make_uint2(words[0], words[1]);
}

// CTA (run of step tokens, kv head, 0 keys / 1 values); a thread takes sixteen
// elements of a head in each pass, so that what a group needs once (its range,
// two divisions, two roundings) is done by four lanes and not eight, and has
// all its loads in flight at the start. 14593 tokens of 8 kv heads of 128 dims:
// 22.9 us, 3.3 TB/s; 8 elements a thread and two batches of loads 28.6. Bound by
// its instructions, about 17 per element, and by their standing in line with
// the loads: with the quantising taken out it is 13.3 us.
template <int DIM>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvArgs a, const uint16_t* k, long long ks,
                                                             const uint16_t* v, long long vs) {
  constexpr int W = DIM / 16, kPass = kThreads / W;  // threads of a head; tokens of one pass over the threads
  constexpr int kPasses = kRun<DIM> / kPass;
  __shared__ long long rows[kRun<DIM>];
  const int h = blockIdx.y, which = blockIdx.z;
  const int i0 = blockIdx.x * kRun<DIM>, n = min(kRun<DIM>, a.n_tokens - i0);
  const int w = threadIdx.x % W, t0 = threadIdx.x / W;
  const long long stride = which ? vs : ks;
  const uint16_t* src = (which ? v : k) + i0 * stride + h * DIM + w * 16;
  uint32_t* codes = which ? a.codes[1] : a.codes[0];
  uint16_t* scales = which ? a.scales[1] : a.scales[0];
  uint16_t* biases = which ? a.biases[1] : a.biases[0];
  uint4 x[kPasses][2];
#pragma unroll
  for (int j = 0; j < kPasses; ++j) {  // before the slots are looked up
    const int t = t0 + j * kPass;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      x[j][i] = t < n ? *reinterpret_cast<const uint4*>(src + t * stride + 8 * i) : make_uint4(0, 0, 0, 0);
  }
  token_rows(a, i0, n, h, rows);
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kPasses; ++j) {
    const int t = t0 + j * kPass;
    const long long row = t < n ? rows[t] : -1;
    if (row < 0) continue;  // (the lanes of a group alike)
    uint16_t s, b;
    const uint2 word = quantise16(x[j], &s, &b, &bad);
    *reinterpret_cast<uint2*>(codes + row * (DIM / 8) + 2 * w) = word;
    if ((w & 3) == 0) {
      scales[row * (DIM / 64) + w / 4] = s;
      biases[row * (DIM / 64) + w / 4] = b;
    }
  }
  if (bad) report(a.hdr, MOE_ERR_DEVICE_CHECK, kKvBadNumber);
}

// CTA (run of step tokens, kv head, 0 keys / 1 values), a code word per thread
// and pass, eight passes' loads in flight. Bound by memory: 131072 tokens of 2
// kv heads of 256 dims, 344 MB, 57.5 us, 0.88 of the measured copy rate.
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
