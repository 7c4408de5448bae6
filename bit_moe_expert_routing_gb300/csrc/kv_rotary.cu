// Norms of queries and keys for each head, the rotation to their positions and
// the append to the 4-bit cache, in one pass over a projection's output.
//
//   y = x rsqrt(mean x^2 + eps) w,  (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)
//
// Memory is the floor: a query element is read and written once (4 bytes), a
// key's or value's read (2) and stored (0.5625). So a thread holds sixteen
// elements of a head, the two chunks of eight whose elements are turned
// together, and nothing but a norm's sum and a key's re-ordering leaves its
// registers; the angles, which all heads of a token share, are made once per
// CTA.
#include "kv_host.cuh"
#include "kv_quant.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRun = 16;  // step tokens of a CTA, at most

struct RotaryArgs {
  KvArgs kv;
  const uint64_t* turns;
  const uint8_t* axis;
  const int32_t* positions;
  const float* weight[2];  // queries', keys'
  float eps;
  int half, interleaved, axes;
  int heads;
  const uint16_t* src[3];  // queries, keys, values
  long long stride[3];
  uint16_t* q_out;
  int run, part;  // step tokens of a CTA; of their heads + 2 kv_heads heads
};

// cos and sin of `pos` times `turns` / 2^64 turns: whole turns fall out of the
// 64-bit product, what is left is rounded to 2^-25 of a turn at most.
__device__ __forceinline__ float2 turned_by(uint64_t turns, int pos) {
  const uint64_t angle = turns * uint64_t(int64_t(pos));
  float2 cs;
  sincospif(float(int32_t(angle >> 32)) * 0x1p-31f, &cs.y, &cs.x);
  return cs;
}

// A thread's sixteen elements as fp32.
struct Sixteen {
  float v[2][8];
};
__device__ __forceinline__ Sixteen widen(const uint4 (&x)[2]) {
  Sixteen y;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) y.v[i][2 * j] = bf16lo(w[j]), y.v[i][2 * j + 1] = bf16hi(w[j]);
  }
  return y;
}
__device__ __forceinline__ uint4 narrow(const float (&v)[8]) {
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// 1 / sqrt(mean of the head's squares + eps); W neighbouring lanes hold a head.
template <int W>
__device__ __forceinline__ float inverse_norm(const Sixteen& x, float eps, unsigned lanes) {
  auto sum = [&](float scale) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(x.v[i][j] * scale, x.v[i][j] * scale, s);
#pragma unroll
    for (int off = W / 2; off; off >>= 1) s += __shfl_xor_sync(lanes, s, off);
    return s;
  };
  const float s = sum(1.f);
  if (s < INFINITY) return rsqrtf(s * (1.f / (16 * W)) + eps);
  return rsqrtf(sum(0x1p-70f) * (1.f / (16 * W))) * 0x1p-70f;  // squares past fp32: eps is nothing beside them
}

// CTA (run of step tokens, part of their heads): the queries', the keys', the
// values' heads in turn, W threads to a head.
template <int DIM>
__global__ void __launch_bounds__(kThreads) kv_append_rotary_kernel(const RotaryArgs r) {
  constexpr int W = DIM / 16, kRows = kThreads / W;
  extern __shared__ float2 cs[];  // [run][half]
  __shared__ int pos[kMaxRun], page[kMaxRun];
  const KvArgs& a = r.kv;
  const int i0 = blockIdx.x * r.run, n = min(r.run, a.n_tokens - i0);
  const int h0 = blockIdx.y * r.part, h1 = min(h0 + r.part, r.heads + 2 * a.kv_heads);
  const int w = threadIdx.x % W, row = threadIdx.x / W;
  const unsigned lanes = (W == 32 ? ~0u : (1u << W) - 1u) << (threadIdx.x & 31 & ~(W - 1));

  if (threadIdx.x < n) {
    const int i = i0 + threadIdx.x, b = kv_seq_of(a, i);
    const int p = a.kv_len[b] - (a.q_off[b + 1] - i);
    int pg = -1;
    if (p >= a.max_kv) {
      report(a.hdr, MOE_ERR_DEVICE_CHECK, kKvBadBatch);
    } else if (p >= 0 && h1 > r.heads) {
      const long long first = kv_page_row(a, b, p >> a.page_bits, 0);
      if (first >= 0) pg = int((first >> a.page_bits) / a.kv_heads);
    }
    pos[threadIdx.x] = p;
    page[threadIdx.x] = pg;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < n * r.half; e += kThreads) {
    const int t = e / r.half, f = e - t * r.half;
    int p = pos[t];
    if (r.positions) {
      const int ax = r.axis ? r.axis[f] : 0;
      p = r.positions[(long long)(ax < r.axes ? ax : 0) * a.n_tokens + i0 + t];
    }
    cs[e] = turned_by(r.turns[f], p);
  }
  __syncthreads();

  // this thread's chunks of eight elements: those turned together (halves apart, or neighbours)
  const int pairs = r.half / 8;  // lanes that turn theirs
  const int c0 = r.interleaved || w >= pairs ? 2 * w : w, c1 = r.interleaved || w >= pairs ? 2 * w + 1 : w + pairs;
  bool bad = false;
#pragma unroll
  for (int kind = 0; kind < 3; ++kind) {
    const int first = kind == 0 ? 0 : r.heads + (kind - 1) * a.kv_heads;  // of the kind's heads
    const int lo = max(h0 - first, 0), hi = min(h1 - first, kind == 0 ? r.heads : a.kv_heads);
    const int per = hi - lo;
    if (per <= 0) continue;
    const float* weight = kind < 2 ? r.weight[kind] : nullptr;
    float wt[2][8];
    if (weight)
#pragma unroll
      for (int j = 0; j < 8; ++j) wt[0][j] = weight[8 * c0 + j], wt[1][j] = weight[8 * c1 + j];
    for (int e = row; e < n * per; e += kRows) {
      const int t = e / per, h = lo + e - t * per;
      const uint16_t* src = r.src[kind] + (i0 + t) * r.stride[kind] + h * DIM;
      uint4 x[2];
      if (kind == 2) {
        x[0] = *reinterpret_cast<const uint4*>(src + 16 * w);
        x[1] = *reinterpret_cast<const uint4*>(src + 16 * w + 8);
      } else {
        x[0] = *reinterpret_cast<const uint4*>(src + 8 * c0);
        x[1] = *reinterpret_cast<const uint4*>(src + 8 * c1);
        Sixteen y = widen(x);
        if (weight) {
          const float inv = inverse_norm<W>(y, r.eps, lanes);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) y.v[i][j] = y.v[i][j] * inv * wt[i][j];
        }
        if (w < pairs) {
          const float2* at = cs + t * r.half + 8 * w;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 c = at[j];
            float& p = r.interleaved ? y.v[j / 4][2 * (j % 4)] : y.v[0][j];
            float& q = r.interleaved ? y.v[j / 4][2 * (j % 4) + 1] : y.v[1][j];
            const float u = p * c.x - q * c.y;
            q = q * c.x + p * c.y;
            p = u;
          }
        }
        x[0] = narrow(y.v[0]);
        x[1] = narrow(y.v[1]);
      }
      if (kind == 0) {
        uint16_t* dst = r.q_out + ((long long)(i0 + t) * r.heads + h) * DIM;
        *reinterpret_cast<uint4*>(dst + 8 * c0) = x[0];
        *reinterpret_cast<uint4*>(dst + 8 * c1) = x[1];
        continue;
      }
      if (kind == 1 && !r.interleaved) {
        // the quantisation takes a head's elements in order: chunks 2 w and 2 w + 1, from where they are
        uint4 z[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = 2 * w + i;
          const int from = c < pairs ? c : c < 2 * pairs ? c - pairs : c / 2;
          const bool second = c < pairs ? false : c < 2 * pairs ? true : c & 1;
          auto take = [&](uint32_t u0, uint32_t u1) {
            const uint32_t v0 = __shfl_sync(lanes, u0, from, W), v1 = __shfl_sync(lanes, u1, from, W);
            return second ? v1 : v0;
          };
          z[i] = make_uint4(take(x[0].x, x[1].x), take(x[0].y, x[1].y), take(x[0].z, x[1].z), take(x[0].w, x[1].w));
        }
        x[0] = z[0], x[1] = z[1];
      }
      if (page[t] < 0) continue;
      const long long at = (((long long)page[t] * a.kv_heads + h) << a.page_bits) + (pos[t] & ((1 << a.page_bits) - 1));
      uint16_t s, b;
      const uint2 word = quantise16(x, &s, &b, &bad);
      *reinterpret_cast<uint2*>(a.codes[kind - 1] + at * (DIM / 8) + 2 * w) = word;
      if ((w & 3) == 0) {
        a.scales[kind - 1][at * (DIM / 64) + w / 4] = s;
        a.biases[kind - 1][at * (DIM / 64) + w / 4] = b;
      }
    }
  }
  if (bad) report(a.hdr, MOE_ERR_DEVICE_CHECK, kKvBadNumber);
}

template <int DIM>
cudaError_t launch(RotaryArgs r, const KvCall& c) {
  const int heads = r.heads + 2 * r.kv.kv_heads;
  r.run = kMaxRun;
  r.part = heads;
  const dim3 grid((r.kv.n_tokens + r.run - 1) / r.run, (heads + r.part - 1) / r.part);
  kv_append_rotary_kernel<DIM><<<grid, kThreads, r.run * r.half * sizeof(float2), c.stream>>>(r);
  return c.launched("kv_append_rotary");
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_kv_append_rotary(const moe_kv_cache* cache, const moe_kv_batch* batch, const moe_rotary* rot,
                                           int heads, const uint16_t* q, long long q_stride, uint16_t* q_out,
                                           const uint16_t* k, long long k_stride, const uint16_t* v, long long v_stride,
                                           void* stream) {
  RotaryArgs r{};
  reset_launch_count();
  if (moe_status s = make_args(cache, batch, &r.kv)) return s;
  if (!rot) return MOE_ERR_ARG;
  if (rot->rotary_dim < 0 || rot->rotary_dim > r.kv.dim || rot->rotary_dim % 16) return MOE_ERR_SHAPE;
  if (heads < 1 || heads > 16384 || rot->axes < 1 || rot->axes > 4) return MOE_ERR_SHAPE;
  if (rot->rotary_dim && (!rot->turns || !aligned(rot->turns, 8))) return MOE_ERR_ARG;
  if (!aligned(rot->positions, 4) || !aligned(rot->q_weight, 16) || !aligned(rot->k_weight, 16)) return MOE_ERR_ARG;
  if ((rot->q_weight || rot->k_weight) && !(rot->eps >= 0x1p-64f && std::isfinite(rot->eps))) return MOE_ERR_ARG;
  if (r.kv.n_tokens == 0) return MOE_OK;
  if (!operand_ok(q, q_stride, heads, r.kv.dim) || !operand_ok(k, k_stride, r.kv.kv_heads, r.kv.dim) ||
      !operand_ok(v, v_stride, r.kv.kv_heads, r.kv.dim))
    return MOE_ERR_ARG;
  if (!q_out || !aligned(q_out, 16) || q_out == q || q_out == k || q_out == v) return MOE_ERR_ARG;
  r.turns = rot->turns;
  r.axis = rot->axis;
  r.positions = rot->positions;
  r.weight[0] = rot->q_weight;
  r.weight[1] = rot->k_weight;
  r.eps = rot->eps;
  r.half = rot->rotary_dim / 2;
  r.interleaved = rot->interleaved != 0;
  r.axes = rot->axes;
  r.heads = heads;
  r.src[0] = q, r.src[1] = k, r.src[2] = v;
  r.stride[0] = q_stride, r.stride[1] = k_stride, r.stride[2] = v_stride;
  r.q_out = q_out;
  const KvCall c = begin_call(stream);
  return status_of(r.kv.dim == 64 ? launch<64>(r, c) : r.kv.dim == 128 ? launch<128>(r, c) : launch<256>(r, c));
}
