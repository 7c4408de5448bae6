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
#include "kv_quant.cuh"

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
