// Attention of a few rows (decode, drafted tokens) over the 4-bit cache.
//
// A row is one query head of one step token; the rows that share a kv head
// share its keys. Reading the cache bounds the work: 0.5625 bytes per cached
// element, each of which is multiplied with every row. The kernel keeps the
// dequantisation and the products in registers:
//
//   S^T[key, row] = K^[key, d] Q^T[d, row]     mma m16n8k16, M = 16 keys, N = 8 rows
//   O^T[d, row]  += V^T[d, key] P^T[key, row]  M = 16 dims, K = 16 keys
//
// With keys (and value dims) on the M side a product of eight rows wastes
// nothing, and a lane's 4-bit words expand straight into its A fragment: no
// dequantised value goes through shared memory. (tcgen05 takes its operands
// from shared or tensor memory, so each expanded value would be written and
// read there once more, for N = 8 columns of use; the warp-level MMA is the
// one that multiplies from registers.) The order of d inside the products is
// free as long as both operands share it, and is chosen so that one mask
// gives two codes of a word: a pair (nibble i, nibble i + 4) per register.
//
// The codes become bf16 without a conversion: the raw bits of an integer
// below 256 are, read as a bf16, that integer times 2^-133 (subnormal and
// first normal binade join). So w & 0x000F000F is the pair (q0, q4) 2^-133, w
// & 0x00F000F0 is (q1, q5) 2^-129, and one fused multiply-add with scale *
// 2^113 (2^109) and bias * 2^-20 gives 2^-20 bf16(scale q + bias), rounded
// once, exactly the cached value. The 2^20 goes into the softmax scale for
// the keys and into the output for the values. (The cache holds magnitudes
// up to 2^16, so scale * 2^113 is finite.)
//
// Work split: a CTA takes (sequence, kv head, group of 8 NT rows, range of
// 32-key tiles), its four warps alternate tiles, each with its own ring of
// bulk copies, so that nothing but the final merge joins the warps. Ranges
// are cut so that the GPU is full; a sequence cut into several leaves fp32
// partial outputs, which attention_combine_kernel joins.
#include <algorithm>

#include "kv.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kTile = 32;   // keys per tile
constexpr int kWarps = 4;

// Shared-memory layout of one ring stage: a tile's codes, scales, biases of
// the keys, then of the values, rows as in the cache.
template <int DIM>
struct Stage {
  static constexpr int kCodes = kTile * DIM / 2;
  static constexpr int kSb = kTile * (DIM / 64) * 2;
  static constexpr int kHalf = kCodes + 2 * kSb;
  static constexpr int kBytes = 2 * kHalf;
};

template <int DIM, int NT>
struct FewCfg {
  static constexpr int kStages = DIM == 64 ? 4 : 3;
  static constexpr int kRows = 8 * NT;
  static constexpr int kSteps = DIM / 16;
  static constexpr bool kQReg = NT * DIM <= 256;  // query fragments in registers; else read from shared memory
  static constexpr int kQBytes = NT * kSteps * 32 * 8;
  static constexpr int kOffRing = kQBytes;
  static constexpr int kOffBar = kOffRing + kWarps * kStages * Stage<DIM>::kBytes;
  static constexpr int kOffMl = kOffBar + kWarps * kStages * 8;       // [warp][row] (max, sum)
  static constexpr int kOffAbort = kOffMl + kWarps * kRows * 8;
  static constexpr int kSmem = kOffAbort + 16;
  // the merge puts two warps' outputs into the ring's place
  static_assert(2 * kRows * DIM * 4 <= kWarps * kStages * Stage<DIM>::kBytes, "merge buffer");
  static constexpr int kMinCtas = NT * DIM <= 128 ? 4 : 2;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}

__device__ __forceinline__ uint32_t fma2(uint32_t q, uint32_t s, uint32_t b) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(q), "r"(s), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
constexpr uint32_t bf16_pow2(int e) { return uint32_t(127 + e) << 7; }
constexpr uint32_t kMulLo = bf16_pow2(113) * 0x10001u;    // scale of a low nibble: 2^-20 / 2^-133
constexpr uint32_t kMulHi = bf16_pow2(109) * 0x10001u;    // of a high nibble
constexpr uint32_t kMulBias = bf16_pow2(-20) * 0x10001u;
constexpr float kUnscale = 1048576.f;                     // 2^20

// Scale and bias of a pair of codes, times the powers above.
struct Sb {
  uint32_t lo, hi, b;
};
__device__ __forceinline__ Sb make_sb(uint32_t s2, uint32_t b2) {
  return Sb{mul2(s2, kMulLo), mul2(s2, kMulHi), mul2(b2, kMulBias)};
}

__device__ __forceinline__ uint32_t lds_u16(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }

// The tiles that a group of rows at positions minpos .. maxpos reads: the
// sink tiles [0, n_sink), then [first, first + n - n_sink).
struct Tiles {
  int n_sink, first, n;
  __device__ __forceinline__ int key0(int t) const { return kTile * (t < n_sink ? t : first + t - n_sink); }
};
__device__ __forceinline__ Tiles tiles_of(int minpos, int maxpos, int window, int sinks) {
  Tiles t{0, 0, 0};
  if (maxpos < 0) return t;
  const int last = maxpos / kTile;  // tile of the last key
  if (window > 0) {
    t.first = max(0, minpos - window + 1) / kTile;
    t.n_sink = min((min(sinks, maxpos + 1) + kTile - 1) / kTile, t.first);
  }
  t.n = t.n_sink + last - t.first + 1;
  return t;
}

struct FewArgs {
  AttnArgs a;
  int max_rows;      // sequences with more rows than this are left to the other kernels
  int row_groups;    // groups of 8 NT rows per (sequence, kv head)
  int chunk;         // tiles per split
  int n_split;       // splits per group, at most
  float* part_o;     // [split][token * heads + head][DIM], normalised
  float* part_lse;   // [split][token * heads + head], base 2
};

// Sizes shared with the combine kernel.
struct Group {
  int n_rows, minpos, maxpos;
  Tiles tiles;
  int splits;
};
__device__ __forceinline__ Group group_of(const FewArgs& f, const SeqInfo& s, int rows_per_group, int rg) {
  Group g;
  const int G = f.a.group, r0 = rg * rows_per_group;
  g.n_rows = min(s.n_new * G - r0, rows_per_group);
  if (s.n_new * G > f.max_rows) g.n_rows = 0;
  if (g.n_rows <= 0) {
    g.n_rows = g.splits = 0;
    return g;
  }
  const int base = s.kv - s.n_new;
  g.minpos = base + r0 / G;
  g.maxpos = base + (r0 + g.n_rows - 1) / G;
  g.tiles = tiles_of(g.minpos, g.maxpos, f.a.window, f.a.sinks);
  g.splits = max(1, (g.tiles.n + f.chunk - 1) / f.chunk);
  return g;
}

template <int DIM, int NT>
__global__ void __launch_bounds__(kWarps * 32, FewCfg<DIM, NT>::kMinCtas) attention_few_kernel(const FewArgs f) {
  using C = FewCfg<DIM, NT>;
  using St = Stage<DIM>;
  constexpr int kSteps = C::kSteps, kStages = C::kStages;
  constexpr int KW = DIM / 32;  // words of a key row that one lane expands (four lanes share a row)
  constexpr int VW = DIM / 64;  // words of a value row per lane (eight lanes share a row)
  extern __shared__ __align__(128) uint8_t smem[];
  const AttnArgs& a = f.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  griddep_launch();

  int x = blockIdx.x;
  const int split = x % f.n_split;
  x /= f.n_split;
  const int rg = x % f.row_groups;
  x /= f.row_groups;
  const int kvh = x % a.kv.kv_heads, b = x / a.kv.kv_heads;
  const SeqInfo si = kv_seq(a.kv, b);
  const Group gr = group_of(f, si, C::kRows, rg);
  if (split >= gr.splits) return;
  const int t_begin = split * f.chunk, t_end = min(gr.tiles.n, t_begin + f.chunk);
  const int lo_all = a.window > 0 ? max(0, gr.minpos - a.window + 1) : 0;  // first windowed key any row sees

  uint8_t* ring = smem + C::kOffRing + warp * kStages * St::kBytes;
  const uint32_t ring_s = smem_u32(ring);
  const uint32_t bar_s = smem_u32(smem + C::kOffBar) + warp * kStages * 8;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffAbort);
  if (lane == 0)
    for (int s = 0; s < kStages; ++s) mbar_init(bar_s + 8 * s, 1);
  if (threadIdx.x == 0) *abort_flag = 0;
  mbar_init_fence();
  __syncwarp();

  // Copies of a tile: one lane per (page piece, array). A piece is the part
  // of the tile in one page: 16 or 32 keys.
  const int piece = a.kv.page_bits < 5 ? 16 : 32;
  const int n_pieces = kTile / piece;
  const int my_piece = lane / 6, my_array = lane % 6;  // array: keys' codes, scales, biases, values' the same
  const bool copier = my_piece < n_pieces;
  // page of this lane's piece of a tile: the table's entry if some row sees a key of the piece, else -1
  auto entry_of = [&](int t) -> int {
    if (!copier || t >= t_end) return -1;
    const int k0 = gr.tiles.key0(t) + my_piece * piece;
    if (k0 > gr.maxpos || (a.window > 0 && k0 + piece <= lo_all && k0 >= a.sinks)) return -1;
    const int j = k0 >> a.kv.page_bits;
    int e = -1;
    if (j < a.kv.table_stride) e = a.kv.table[(long long)b * a.kv.table_stride + j];
    if (e < 0 || e >= a.kv.n_pages) {
      e = -1;
      report(a.kv.hdr, MOE_ERR_DEVICE_CHECK, kKvBadPage);
    }
    return e;
  };
  // array pointers by index arithmetic would index the parameter space: pick once
  const uint8_t* src_base;
  int row_bytes, dst_off;
  {
    const int which = my_array / 3, kind = my_array % 3;
    src_base = kind == 0   ? reinterpret_cast<const uint8_t*>(which ? a.kv.codes[1] : a.kv.codes[0])
               : kind == 1 ? reinterpret_cast<const uint8_t*>(which ? a.kv.scales[1] : a.kv.scales[0])
                           : reinterpret_cast<const uint8_t*>(which ? a.kv.biases[1] : a.kv.biases[0]);
    row_bytes = kind == 0 ? DIM / 2 : DIM / 32;
    dst_off = which * St::kHalf + (kind == 0 ? 0 : St::kCodes + (kind - 1) * St::kSb);
  }
  // Issues tile t into stage s with page entry e (of this lane's piece);
  // returns which pieces are there.
  auto issue = [&](int t, int s, int e) -> unsigned {
    const unsigned have = __ballot_sync(~0u, e >= 0);
    const uint32_t bar = bar_s + 8 * s;
    const int n = __popc(have) / 6;
    if (lane == 0) mbar_arrive_tx(bar, uint32_t(n) * piece * (2 * (DIM / 2) + 4 * (DIM / 32)));
    __syncwarp();
    if (e >= 0) {
      const int k0 = gr.tiles.key0(t) + my_piece * piece;
      const long long row = ((long long)e * a.kv.kv_heads + kvh << a.kv.page_bits) + (k0 & ((1 << a.kv.page_bits) - 1));
      bulk_g2s(ring_s + s * St::kBytes + dst_off + my_piece * piece * row_bytes, src_base + row * row_bytes,
               piece * row_bytes, bar);
    }
    return (have & 1u) | (n_pieces == 2 ? (have >> 5) & 2u : (have & 1u) << 1);  // bit i: keys 16 i .. 16 i + 15
  };
  unsigned there[kStages];
  int nxt = entry_of(t_begin + warp);
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    const int t = t_begin + warp + s * kWarps;
    there[s] = 0;
    if (t < t_end) {
      const int e = nxt;
      nxt = entry_of(t + kWarps);
      there[s] = issue(t, s, e);
    }
  }

  // Query fragments, while the first tiles are on their way: B fragment of
  // step 2 m + h for row n = lane / 4 holds, for word W = KW c + m, dims 8 W +
  // 2 h + {0, 4} and 8 W + 2 h + {1, 5}.
  uint2* qs = reinterpret_cast<uint2*>(smem);
  for (int e = threadIdx.x; e < NT * kSteps * 32; e += kWarps * 32) {
    const int l = e & 31, step = (e >> 5) % kSteps, nt = (e >> 5) / kSteps;
    const int row = 8 * nt + (l >> 2);
    uint2 v = make_uint2(0, 0);
    if (row < gr.n_rows) {
      const int r = rg * C::kRows + row;
      const uint16_t* q = a.q + (si.first + r / a.group) * a.q_stride + (kvh * a.group + r % a.group) * DIM +
                          8 * (KW * (l & 3) + step / 2) + 2 * (step & 1);
      v = make_uint2(q[0] | uint32_t(q[4]) << 16, q[1] | uint32_t(q[5]) << 16);
    }
    qs[e] = v;
  }
  __syncthreads();
  uint2 qr[C::kQReg ? NT : 1][C::kQReg ? kSteps : 1];
  if (C::kQReg) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int s = 0; s < kSteps; ++s) qr[n][s] = qs[(n * kSteps + s) * 32 + lane];
  }

  float o[NT][kSteps][4];  // O^T: [rows' tile][value tile][fragment]
  float m[NT][2], l[NT][2];  // per row 2 c + i of a tile: reference maximum (base 2), this lane's part of the sum
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < 2; ++i) m[n][i] = -INFINITY, l[n][i] = 0.f;
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][j][i] = 0.f;
  }
  const float to_log2 = a.scale * (1.4426950408889634f * kUnscale);
  // Key of fragment index i (0..15) in a 16-key half of a tile: the two rows
  // of each pair swap for every other pair, which spreads both the key and
  // the value reads over the shared-memory banks.
  const int krow = 2 * (g >> 1) + ((g & 1) ^ ((g >> 1) & 1));
  const int vrow0 = 2 * c + (c & 1), vrow1 = 2 * c + ((c & 1) ^ 1);

  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int t = t_begin + warp; t < t_end; t += kWarps) {
    if (!(ok = mbar_wait(bar_s + 8 * stage, phase, abort_flag, a.kv.hdr, kWaitLimit, false, 210))) break;
    unsigned have = 0;
#pragma unroll
    for (int s = 0; s < kStages; ++s)
      if (s == stage) have = there[s];
    const uint8_t* kc = ring + stage * St::kBytes;
    const uint8_t* vc = kc + St::kHalf;
    const int k0 = gr.tiles.key0(t);
    const bool whole = have == 3 && k0 + kTile - 1 <= gr.minpos &&
                       (a.window == 0 || k0 > gr.maxpos - a.window || k0 + kTile <= a.sinks);

    // scores
    float sc[NT][2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][u][i] = 0.f;
      uint32_t w[2][KW];
      Sb sb[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * u + 8 * h + krow;
        const uint32_t* p = reinterpret_cast<const uint32_t*>(kc + row * (DIM / 2)) + KW * c;
        if (KW == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          w[h][0] = v.x, w[h][1] = v.y;
        } else {
#pragma unroll
          for (int q = 0; q < KW; q += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + q);
            w[h][q] = v.x, w[h][q + 1] = v.y, w[h][(q + 2) % KW] = v.z, w[h][(q + 3) % KW] = v.w;
          }
        }
        const uint8_t* ps = kc + St::kCodes + (row * (DIM / 64) + (c * KW) / 8) * 2;
        sb[h] = make_sb(lds_u16(ps) * 0x10001u, lds_u16(ps + St::kSb) * 0x10001u);
      }
#pragma unroll
      for (int j = 0; j < KW; ++j) {
        uint32_t p[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t v = w[h][j], v8 = v >> 8;
          p[h][0] = fma2(v & 0x000F000Fu, sb[h].lo, sb[h].b);
          p[h][1] = fma2(v & 0x00F000F0u, sb[h].hi, sb[h].b);
          p[h][2] = fma2(v8 & 0x000F000Fu, sb[h].lo, sb[h].b);
          p[h][3] = fma2(v8 & 0x00F000F0u, sb[h].hi, sb[h].b);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma(sc[n][u], p[0][2 * h], p[1][2 * h], p[0][2 * h + 1], p[1][2 * h + 1],
                C::kQReg ? qr[C::kQReg ? n : 0][C::kQReg ? 2 * j + h : 0] : qs[(n * kSteps + 2 * j + h) * 32 + lane]);
      }
    }
    // base-2 scores; what a row does not see is -inf
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][u][i] *= to_log2;
    if (!whole) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int pos = si.kv - si.n_new + (rg * C::kRows + 8 * n + 2 * c + i) / a.group;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int key = k0 + 16 * u + 8 * h + krow;
              const bool sees = ((have >> u) & 1u) && key <= pos &&
                                (a.window == 0 || key > pos - a.window || key < a.sinks);
              if (!sees) sc[n][u][2 * h + i] = -INFINITY;
            }
        }
    }
    // running maximum: the reference moves only when a score passes it by 2^8, which costs no precision (the
    // probabilities are floating point) and leaves most tiles without a rescaling
    float mx[NT][2];
    bool grew = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = fmaxf(fmaxf(sc[n][0][i], sc[n][0][2 + i]), fmaxf(sc[n][1][i], sc[n][1][2 + i]));
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, off));
        mx[n][i] = v;
        grew |= v > m[n][i] + 8.f;
      }
    if (__any_sync(~0u, grew)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float al[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float v = fmaxf(m[n][i], mx[n][i]);
          al[i] = v == -INFINITY ? 1.f : ex2(m[n][i] - v);
          m[n][i] = v;
          l[n][i] *= al[i];
        }
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          o[n][j][0] *= al[0], o[n][j][1] *= al[1];
          o[n][j][2] *= al[0], o[n][j][3] *= al[1];
        }
      }
    }
    // probabilities; transposed to the B fragments of the value product
    uint2 pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float r0 = m[n][0] == -INFINITY ? 0.f : m[n][0], r1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float* s = sc[n][u];
        s[0] = ex2(s[0] - r0), s[1] = ex2(s[1] - r1), s[2] = ex2(s[2] - r0), s[3] = ex2(s[3] - r1);
        l[n][0] += s[0] + s[2], l[n][1] += s[1] + s[3];
        uint32_t h0, h1;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h0) : "f"(s[1]), "f"(s[0]));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h1) : "f"(s[3]), "f"(s[2]));
        asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pb[n][u].x) : "r"(h0));
        asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pb[n][u].y) : "r"(h1));
      }
    }
    // values
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t w[4][VW];
      uint32_t ss[4], bb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // keys of fragment indexes 2 c, 2 c + 1, 2 c + 8, 2 c + 9
        const int row = 16 * u + 8 * (i >> 1) + ((i & 1) ? vrow1 : vrow0);
        const uint32_t* p = reinterpret_cast<const uint32_t*>(vc + row * (DIM / 2)) + VW * g;
        if (VW == 1) {
          w[i][0] = *p;
        } else if (VW == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          w[i][0] = v.x, w[i][VW - 1] = v.y;
        } else {
          const uint4 v = *reinterpret_cast<const uint4*>(p);
          w[i][0] = v.x, w[i][1 % VW] = v.y, w[i][2 % VW] = v.z, w[i][3 % VW] = v.w;
        }
        const uint8_t* ps = vc + St::kCodes + (row * (DIM / 64) + (g * VW) / 8) * 2;
        ss[i] = lds_u16(ps), bb[i] = lds_u16(ps + St::kSb);
        if (!whole) {  // a slot that no row sees may hold anything: its zero probability needs a finite value
          const int key = k0 + row;
          const bool used = ((have >> u) & 1u) && key <= gr.maxpos &&
                            (a.window == 0 || key >= lo_all || key < a.sinks);
          if (!used) ss[i] = bb[i] = 0;
        }
      }
      Sb sb[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) sb[h] = make_sb(ss[2 * h] | ss[2 * h + 1] << 16, bb[2 * h] | bb[2 * h + 1] << 16);
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        uint32_t v[2][4];  // byte k of the pair's two words, in bits 0..7 and 16..23
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w0 = w[2 * h][j], w1 = w[2 * h + 1][j];
          v[h][0] = __byte_perm(w0, w1, 0x5410);
          v[h][1] = v[h][0] >> 8;
          v[h][2] = __byte_perm(w0, w1, 0x7632);
          v[h][3] = v[h][2] >> 8;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a0 = fma2(v[0][k] & 0x000F000Fu, sb[0].lo, sb[0].b);
          const uint32_t a1 = fma2(v[0][k] & 0x00F000F0u, sb[0].hi, sb[0].b);
          const uint32_t a2 = fma2(v[1][k] & 0x000F000Fu, sb[1].lo, sb[1].b);
          const uint32_t a3 = fma2(v[1][k] & 0x00F000F0u, sb[1].hi, sb[1].b);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma(o[n][4 * j + k], a0, a1, a2, a3, pb[n][u]);
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    {
      const int tn = t + kStages * kWarps;
      unsigned h = 0;
      if (tn < t_end) {
        const int e = nxt;
        nxt = entry_of(tn + kWarps);
        h = issue(tn, stage, e);
      }
#pragma unroll
      for (int s = 0; s < kStages; ++s)
        if (s == stage) there[s] = h;
    }
    if (++stage == kStages) stage = 0, phase ^= 1;
  }
  if (!ok) {  // a wait gave up: the copies in flight may still land, wait for each again (bounded) before leaving
    for (int s = 0; s < kStages; ++s) mbar_wait(bar_s + 8 * s, s < stage ? phase ^ 1 : phase, abort_flag, a.kv.hdr, kWaitLimit, true, 211);
  }

  // Merge of the four warps: sums over the lanes that share a row, then the
  // outputs of warps 2, 3 into 0, 1 and of 1 into 0 (two buffers in the ring).
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int off = 4; off <= 16; off <<= 1) l[n][i] += __shfl_xor_sync(~0u, l[n][i], off);
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
  if (g == 0)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) ml[warp * C::kRows + 8 * n + 2 * c + i] = make_float2(m[n][i], l[n][i]);
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float fac[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = -INFINITY, sum = 0.f;
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * C::kRows + 8 * n + 2 * c + i].x);
      const float ref = top == -INFINITY ? 0.f : top;
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = ml[w * C::kRows + 8 * n + 2 * c + i];
        sum += ex2(v.x - ref) * v.y;
      }
      // kUnscale: the values' 2^-20
      fac[i] = sum != 0.f ? ex2(m[n][i] - ref) / sum * kUnscale : 0.f;
      l[n][i] = sum != 0.f ? top + log2f(sum) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      o[n][j][0] *= fac[0], o[n][j][1] *= fac[1];
      o[n][j][2] *= fac[0], o[n][j][3] *= fac[1];
    }
  }
  float* buf = reinterpret_cast<float*>(smem + C::kOffRing);
  // fragment (j = 4 word + k) of lane (g, c): dims 8 (VW g + word) + 2 k + {0, 1} of rows 2 c, 2 c + 1
  auto each = [&](auto&& fn) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int d = 8 * (VW * g + j / 4) + 2 * (j % 4);
        fn(8 * n + 2 * c, d, o[n][j][0], o[n][j][2]);
        fn(8 * n + 2 * c + 1, d, o[n][j][1], o[n][j][3]);
      }
  };
#pragma unroll
  for (int from = 2; from >= 1; from >>= 1) {
    if (warp >= from && warp < 2 * from)
      each([&](int r, int d, float& x0, float& x1) {
        *reinterpret_cast<float2*>(buf + ((warp - from) * C::kRows + r) * DIM + d) = make_float2(x0, x1);
      });
    __syncthreads();
    if (warp < from)
      each([&](int r, int d, float& x0, float& x1) {
        const float2 v = *reinterpret_cast<const float2*>(buf + (warp * C::kRows + r) * DIM + d);
        x0 += v.x, x1 += v.y;
      });
    __syncthreads();
  }
  if (warp == 0)
    each([&](int r, int d, float& x0, float& x1) {
      *reinterpret_cast<float2*>(buf + r * DIM + d) = make_float2(x0, x1);
    });
  if (warp == 0 && g == 0)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) ml[8 * n + 2 * c + i].x = l[n][i];
  __syncthreads();
  const long long all_rows = (long long)a.kv.n_tokens * a.heads;
  for (int e = threadIdx.x; e < gr.n_rows * (DIM / 4); e += kWarps * 32) {
    const int row = e / (DIM / 4), d = e % (DIM / 4) * 4;
    const int r = rg * C::kRows + row;
    const long long at = (long long)(si.first + r / a.group) * a.heads + kvh * a.group + r % a.group;
    const float4 v = *reinterpret_cast<const float4*>(buf + row * DIM + d);
    const float lse = ml[row].x;
    if (gr.splits == 1) {
      uint2 w;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(v.y), "f"(v.x));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(v.w), "f"(v.z));
      *reinterpret_cast<uint2*>(a.out + at * DIM + d) = w;
      if (d == 0 && a.lse) a.lse[at] = lse * 0.6931471805599453f;
    } else {
      *reinterpret_cast<float4*>(f.part_o + (split * all_rows + at) * DIM + d) = v;
      if (d == 0) f.part_lse[split * all_rows + at] = lse;
    }
  }
}

// Joins the splits of a row: out = sum_s 2^(lse_s - max) o_s / sum_s 2^(lse_s
// - max). One CTA of eight warps per (sequence, kv head, row that the kernel
// above may take); a warp takes every eighth split.
template <int DIM>
__global__ void __launch_bounds__(256) attention_combine_kernel(const FewArgs f, int rows_per_group, int rows_max) {
  __shared__ float acc[8][DIM];
  __shared__ float2 ms[8];
  const AttnArgs& a = f.a;
  const int r = blockIdx.x % rows_max, kvh = blockIdx.x / rows_max % a.kv.kv_heads, b = blockIdx.x / rows_max / a.kv.kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqInfo si = kv_seq(a.kv, b);
  const Group gr = group_of(f, si, rows_per_group, r / rows_per_group);
  if (gr.splits <= 1 || r % rows_per_group >= gr.n_rows) return;
  griddep_wait();
  const long long at = (long long)(si.first + r / a.group) * a.heads + kvh * a.group + r % a.group;
  const long long all_rows = (long long)a.kv.n_tokens * a.heads;
  float top = -INFINITY;
  for (int s = lane; s < gr.splits; s += 32) top = fmaxf(top, f.part_lse[s * all_rows + at]);
#pragma unroll
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, off));
  const float ref = top == -INFINITY ? 0.f : top;
  float o[DIM / 32], sum = 0.f;
#pragma unroll
  for (int j = 0; j < DIM / 32; ++j) o[j] = 0.f;
  for (int s = warp; s < gr.splits; s += 8) {
    const float w = ex2(f.part_lse[s * all_rows + at] - ref);
    sum += w;
    const float* p = f.part_o + (s * all_rows + at) * DIM;
#pragma unroll
    for (int j = 0; j < DIM / 32; ++j) o[j] += w * p[lane + 32 * j];
  }
#pragma unroll
  for (int j = 0; j < DIM / 32; ++j) acc[warp][lane + 32 * j] = o[j];
  if (lane == 0) ms[warp].x = sum;
  __syncthreads();
  float tot = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) tot += ms[w].x;
  const int d = threadIdx.x;
  if (d < DIM) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += acc[w][d];
    a.out[at * DIM + d] = f32_to_bf16(tot != 0.f ? v / tot : 0.f);
  }
  if (d == 0 && a.lse) a.lse[at] = tot != 0.f ? (top + log2f(tot)) * 0.6931471805599453f : -INFINITY;
}

// Host plan: rows per group (from the most rows a sequence can have), tiles
// per split and their number.
struct FewPlan {
  int nt, row_groups, chunk, n_split;
  size_t part_rows;
};

FewPlan plan(const AttnArgs& a, int max_rows) {
  FewPlan p;
  const long long rows = std::min<long long>((long long)a.kv.max_new * a.group, max_rows);
  p.nt = rows <= 8 ? 1 : rows <= 16 || a.kv.dim == 256 ? 2 : 4;
  p.row_groups = int((rows + 8 * p.nt - 1) / (8 * p.nt));
  long long keys = a.kv.max_kv;
  if (a.window > 0) keys = std::min<long long>(keys, (long long)a.window + std::min(a.sinks, a.kv.max_kv) + a.kv.max_new + 2 * kTile);
  const int tiles = std::max(1, int((keys + kTile - 1) / kTile));
  // enough splits to give every SM a few CTAs, none shorter than two tiles
  // per warp
  const long long items = std::max(1ll, (long long)a.kv.n_seqs * a.kv.kv_heads * p.row_groups);
  const int per_sm = a.kv.dim == 256 || p.nt > 1 ? 2 : 4;
  const long long want = std::max(1ll, (long long)num_sms() * per_sm / items);
  int chunk = int((tiles + want - 1) / want);
  chunk = std::max(chunk, 2 * kWarps);
  chunk = std::min(chunk, 32);
  chunk = (chunk + kWarps - 1) / kWarps * kWarps;
  p.chunk = chunk;
  p.n_split = (tiles + chunk - 1) / chunk;
  p.part_rows = p.n_split > 1 ? size_t(p.n_split) * a.kv.n_tokens * a.heads : 0;
  return p;
}

template <int DIM, int NT>
cudaError_t launch(const FewArgs& f, const KvCall& c) {
  using C = FewCfg<DIM, NT>;
  const void* fn = reinterpret_cast<const void*>(&attention_few_kernel<DIM, NT>);
  if (!ensure_smem_limit(fn, C::kSmem)) return cudaErrorInvalidValue;
  const long long grid = 1ll * f.n_split * f.row_groups * f.a.kv.kv_heads * f.a.kv.n_seqs;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  attention_few_kernel<DIM, NT><<<unsigned(grid), kWarps * 32, C::kSmem, c.stream>>>(f);
  if (cudaError_t e = c.launched("attention_few")) return e;
  if (f.n_split == 1) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  const int rows_max = int(std::min<long long>((long long)f.a.kv.max_new * f.a.group, f.max_rows));
  const long long rows = 1ll * rows_max * f.a.kv.kv_heads * f.a.kv.n_seqs;
  if (rows > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(unsigned(rows));
  cfg.blockDim = dim3(256);
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, attention_combine_kernel<DIM>, f, C::kRows, rows_max)) return e;
  return c.launched("attention_combine");
}

}  // namespace

size_t attention_few_workspace(const AttnArgs& a, int max_rows) {
  const FewPlan p = plan(a, max_rows);
  return p.part_rows * (size_t(a.kv.dim) + 1) * 4;
}

cudaError_t attention_few(const AttnArgs& a, int max_rows, void* ws, const KvCall& c) {
  const FewPlan p = plan(a, max_rows);
  float* part = static_cast<float*>(ws);
  const FewArgs f{a, max_rows, p.row_groups, p.chunk, p.n_split, part, part + p.part_rows * a.kv.dim};
  switch (a.kv.dim * 8 + p.nt) {
    case 64 * 8 + 1: return launch<64, 1>(f, c);
    case 64 * 8 + 2: return launch<64, 2>(f, c);
    case 64 * 8 + 4: return launch<64, 4>(f, c);
    case 128 * 8 + 1: return launch<128, 1>(f, c);
    case 128 * 8 + 2: return launch<128, 2>(f, c);
    case 128 * 8 + 4: return launch<128, 4>(f, c);
    case 256 * 8 + 1: return launch<256, 1>(f, c);
    default: return launch<256, 2>(f, c);
  }
}

}  // namespace moe
