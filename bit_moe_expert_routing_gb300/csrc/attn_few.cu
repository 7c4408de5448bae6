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
// 2^110 (2^106) and bias * 2^-23 gives 2^-23 bf16(scale q + bias), rounded
// once: exactly the cached value, but that a value or bias below 2^-103 is
// rounded to a multiple of 2^-110. The 2^23 goes into the softmax scale for the keys and
// into the output for the values. (A smaller power would hold smaller values
// exactly and overflow on scales below 2^18: a cache's magnitudes of at most
// 2^16 can come of scales up to 2^17.)
//
// Work split: an item is (sequence, kv head, group of 8 NT rows), and its
// units are its 32-key tiles. One wave of CTAs takes equal, contiguous ranges
// of all items' units, whatever the sequences' lengths; an item that is cut
// leaves fp32 partial outputs, which a combine kernel joins. (A grid of
// fixed-length splits took 107 us for 64 ragged sequences of up to 8191
// positions, 60 of them in prologues and merges.) When no item has more than
// whole_keys, an item is a CTA's whole work and nothing is cut. The four warps
// of a CTA alternate tiles, each with its own ring of asynchronous copies, so
// that nothing but the merge of an item's end joins them. (cp.async rather than
// bulk copies: a tile is six runs of one or two pages, and six bulk copies by
// six lanes take the warp 1200 cycles to issue.)
//
// Measured, calls replayed from a graph: 64 sequences of 700 to 8191 positions,
// 32 heads over 8 of 128 dims, 70 us for 324 MB, 4.6 TB/s: bound by issue slots
// and the ALU, some 630 warp instructions per tile, of which 288 expand codes
// and 48 multiply. (With the table's entries looked up per tile, not per 32
// tiles, 75 us.) One sequence at 65537, 16 heads over 2 of 256 dims: 18 us for
// 37 MB, 3.4 tiles per warp, bound by the chain of its first loads and the join.
// 32 sequences with a window of 1024, heads of 64, 8 kv heads: 10.5 us for 19 MB in
// 256 whole items, one or two to an SM, nine tiles per warp one after the other:
// issue slots 37% of the active cycles, SMs active in 69% of the time.
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
  static constexpr int kQBytes = kQReg ? 0 : NT * kSteps * 32 * 8;
  static constexpr int kOffRing = kQBytes;
  static constexpr int kOffMl = kOffRing + kWarps * kStages * Stage<DIM>::kBytes;  // [warp][row] (max, sum)
  static constexpr int kSmem = kOffMl + kWarps * kRows * 8;
  // the merge puts three warps' outputs into the ring's place
  static_assert(3 * kRows * DIM * 4 <= kWarps * kStages * Stage<DIM>::kBytes, "merge buffer");
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
constexpr uint32_t kMulLo = bf16_pow2(110) * 0x10001u;    // scale of a low nibble: 2^-23 / 2^-133
constexpr uint32_t kMulHi = bf16_pow2(106) * 0x10001u;    // of a high nibble
constexpr uint32_t kMulBias = bf16_pow2(-23) * 0x10001u;
constexpr float kUnscale = 8388608.f;                     // 2^23

// Scale and bias of a pair of codes, times the powers above.
struct Sb {
  uint32_t lo, hi, b;
};
__device__ __forceinline__ Sb make_sb(uint32_t s2, uint32_t b2) {
  return Sb{mul2(s2, kMulLo), mul2(s2, kMulHi), mul2(b2, kMulBias)};
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

// Items of at most so many keys are not worth cutting: the combine kernel and
// the parts cost more than the tiles that an item's CTA would be spared. With
// more items less is spared, since the CTAs that would share them have items
// of their own. (Cut against whole, us, one token per sequence; heads of 64, 4
// kv heads: 1 sequence 600 keys 7.5 and 6.8, 1000 keys 7.5 and 8.3; 32
// sequences 1500 keys 11.8 and 10.4, 2200 keys 13.6 and 13.7. Heads of 128, 2
// kv heads: 8 sequences 600 keys 9.7 and 7.9, 1000 keys 9.9 and 10.1; 64
// sequences 1500 keys 15.1 and 13.0, 2200 keys 17.9 and 17.1. Heads of 256: 1
// sequence 256 keys 9.6 and 7.5, 600 keys 9.6 and 10.8; 64 sequences 1500 keys
// 20.0 and 18.7.) The bound on the lengths is all that is known here, and
// shorter sequences gain from a cut, so not above 2048.
long long whole_keys(int dim, long long items) {
  return std::min(2048ll, std::max(dim == 256 ? 448ll : 896ll, 16 * items));
}
constexpr int kMinTiles = 8;  // of a CTA, when items are cut: two per warp
// What beginning, merging and writing an item costs a CTA, in tiles: counted
// in front of its tiles when units are dealt out. (64 ragged sequences, 512
// items: CTAs with four items took 143 thousand cycles, with one 112.)
constexpr int kItemCost = 10;

struct FewArgs {
  AttnArgs a;
  int max_rows;      // sequences with more rows than this are left to the other kernels
  int row_groups;    // groups of 8 NT rows per (sequence, kv head), at most
  int whole;         // every CTA takes one item, whole
  int max_ctas;      // else: CTAs of the grid
  float* part_o;     // [2 max_ctas][8 NT][DIM], normalised
  float* part_lse;   // [2 max_ctas][8 NT], base 2
  unsigned long long inv_group;  // ceil(2^32 / group): row / group for the rows of a sequence
  __device__ __forceinline__ int token(int row) const { return int((unsigned(row) * inv_group) >> 32); }
};

// A sequence as its items: `groups` per kv head, each with kItemCost +
// `tiles.n` units (the sequence's tiles; a row group that sees fewer masks the
// rest).
struct SeqItems {
  SeqInfo s;
  int groups, rows;  // row groups of a kv head, rows of all of them
  Tiles tiles;
  __device__ __forceinline__ long long units(int kv_heads) const { return (long long)groups * kv_heads * (kItemCost + tiles.n); }
};
__device__ __forceinline__ SeqItems items_of(const FewArgs& f, int b, int rows_per_group) {
  SeqItems q;
  q.s = kv_seq(f.a.kv, b);
  q.rows = q.s.n_new * f.a.group;
  if (q.rows > f.max_rows) q.rows = 0;
  q.groups = (q.rows + rows_per_group - 1) / rows_per_group;
  q.tiles = tiles_of(q.s.kv - q.s.n_new, q.s.kv - 1, f.a.window, f.a.sinks);
  if (q.tiles.n == 0) q.tiles.n = 1;  // rows that see nothing are written too
  return q;
}

// The units of all sequences, and where unit ranges begin. One CTA computes
// it, kScanThreads sequences at a time.
template <int THREADS>
struct Cut {
  const FewArgs& f;
  const int rows;
  long long* sums;  // [THREADS] shared memory
  long long total, each;
  int ctas, more;

  // prefix sums of the units of sequences c0 .. c0 + THREADS - 1 in `sums`; their total
  __device__ long long chunk(int c0) {
    const int b = c0 + threadIdx.x;
    long long v = b < f.a.kv.n_seqs ? items_of(f, b, rows).units(f.a.kv.kv_heads) : 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long u = __shfl_up_sync(~0u, v, off);
      if (lane >= off) v += u;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp; ++w) before += sums[w];
    __syncthreads();
    sums[threadIdx.x] = v + before;
    __syncthreads();
    return sums[THREADS - 1];
  }
  __device__ Cut(const FewArgs& args, int rows_per_group, long long* shared) : f(args), rows(rows_per_group), sums(shared) {
    total = 0;
    if (f.a.kv.n_seqs == 1) {  // one request: no sums to make
      total = items_of(f, 0, rows).units(f.a.kv.kv_heads);
    } else {
      for (int c0 = 0; c0 < f.a.kv.n_seqs; c0 += THREADS) total += chunk(c0);
    }
    const long long want = (total + kMinTiles - 1) / kMinTiles;
    ctas = int(want < f.max_ctas ? (want > 1 ? want : 1) : f.max_ctas);
    each = total < 0x7fffffff ? unsigned(total) / unsigned(ctas) : total / ctas;
    more = int(total - each * ctas);
  }
  // the first `more` CTAs take each + 1 units, the others `each`
  __device__ long long begin(int c) const { return each * c + min(c, more); }
  __device__ int cta_of(long long u) const {
    const long long split = (each + 1) * more;
    if (total < 0x7fffffff) return u < split ? unsigned(u) / unsigned(each + 1) : more + unsigned(u - split) / unsigned(each);
    return int(u < split ? u / (each + 1) : more + (u - split) / each);
  }
  // sequence that holds unit u < total, and u's place within it
  __device__ int find(long long u, int* at) {
    if (f.a.kv.n_seqs == 1) {
      *at = int(u);
      return 0;
    }
    long long base = 0;
    for (int c0 = 0;; c0 += THREADS) {
      const long long n = f.a.kv.n_seqs <= THREADS ? total : chunk(c0);
      if (u - base < n) {
        int lo = 0, hi = THREADS - 1;  // the first with sums > u - base
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (sums[mid] > u - base)
            hi = mid;
          else
            lo = mid + 1;
        }
        *at = int(u - base - (lo ? sums[lo - 1] : 0));
        return c0 + lo;
      }
      base += n;
    }
  }
};

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
  uint8_t* ring = smem + C::kOffRing + warp * kStages * St::kBytes;
  const uint32_t ring_s = smem_u32(ring);

  // this CTA's units: `left` of them from unit `off` of item `item` of sequence b on
  int b, item, off;
  long long left;
  SeqItems sq;
  if (f.whole) {
    const int per_seq = a.kv.kv_heads * f.row_groups;
    b = blockIdx.x / per_seq;
    const int x = blockIdx.x - b * per_seq, h = x / f.row_groups, r = x - h * f.row_groups;
    sq = items_of(f, b, C::kRows);
    if (r >= sq.groups) return griddep_wait();
    item = h * sq.groups + r;
    off = 0;
    left = kItemCost + sq.tiles.n;
  } else {
    Cut<kWarps * 32> cut(f, C::kRows, reinterpret_cast<long long*>(smem + C::kOffRing));
    if (int(blockIdx.x) >= cut.ctas) return griddep_wait();
    const long long begin = cut.begin(blockIdx.x);
    left = cut.begin(blockIdx.x + 1) - begin;
    if (left <= 0) return griddep_wait();
    int at;  // (launch() sees to it that a sequence has fewer than 2^31 units)
    b = cut.find(begin, &at);
    sq = items_of(f, b, C::kRows);
    item = at / (kItemCost + sq.tiles.n);
    off = at - item * (kItemCost + sq.tiles.n);
    __syncthreads();  // the prefix sums' place becomes the ring's
  }
  while (left > 0) {
  if (item >= sq.groups * a.kv.kv_heads) {  // the next sequence that has items (there is one: units are left)
    item = off = 0;
    do sq = items_of(f, ++b, C::kRows);
    while (sq.groups == 0);
  }
  const int span = int(min((long long)(kItemCost + sq.tiles.n - off), left));
  const int t_begin = max(0, off - kItemCost), t_end = off + span - kItemCost;
  left -= span;
  off = 0;
  if (t_end <= t_begin) {  // none of its tiles
    ++item;
    continue;
  }
  const SeqInfo si = sq.s;
  const int kvh = item / sq.groups, rg = item - kvh * sq.groups;
  struct {
    int n_rows, minpos, maxpos;
    Tiles tiles;
  } gr;
  gr.n_rows = min(sq.rows - rg * C::kRows, C::kRows);
  gr.minpos = si.kv - si.n_new + f.token(rg * C::kRows);
  gr.maxpos = si.kv - si.n_new + f.token(rg * C::kRows + gr.n_rows - 1);
  gr.tiles = sq.tiles;
  const int lo_all = a.window > 0 ? max(0, gr.minpos - a.window + 1) : 0;  // first windowed key any row sees

  // The queries' words for the fragments below, asked for before anything
  // waits: word W = KW c + m of row n = lane / 4 (this warp's share of the
  // words, where the fragments go through shared memory).
  constexpr int kQWords = C::kQReg ? NT * KW : NT * KW / kWarps;
  uint4 qw[kQWords];
#pragma unroll
  for (int e = 0; e < kQWords; ++e) {
    const int x = C::kQReg ? e : e * kWarps + warp, n = x / KW, m = x % KW, row = 8 * n + g;
    qw[e] = make_uint4(0, 0, 0, 0);
    if (row < gr.n_rows) {
      const int r = rg * C::kRows + row, t = f.token(r);
      qw[e] = *reinterpret_cast<const uint4*>(a.q + (si.first + t) * a.q_stride + (kvh * a.group + r - t * a.group) * DIM +
                                              8 * (KW * c + m));
    }
  }

  // Copies of a tile, 16 bytes per lane and instruction, each array's rows in
  // order. Its two halves of 16 keys may lie in different pages. Each lane
  // looks the pages of one of the warp's next 32 tiles up (-1: there is none,
  // recorded, or no row sees a key of that half).
  const bool has_table = a.kv.table_stride > 0;
  const int* table = has_table ? a.kv.table + (long long)b * a.kv.table_stride : a.kv.kv_len;
  const int last_entry = has_table ? a.kv.table_stride - 1 : 0;
  auto pages_of = [&](int n0, int half) -> int {
    const int t = t_begin + warp + kWarps * (n0 + lane);
    const int k0 = gr.tiles.key0(t) + 16 * half, j = k0 >> a.kv.page_bits;
    const int page = __ldg(table + max(0, min(j, last_entry)));
    const bool unseen = (t >= t_end) | (k0 > gr.maxpos) | ((a.window > 0) & (k0 + 16 <= lo_all) & (k0 >= a.sinks));
    const bool bad = (j >= a.kv.table_stride) | (unsigned(page) >= unsigned(a.kv.n_pages));
    if (bad & !unseen) report(a.kv.hdr, MOE_ERR_DEVICE_CHECK, kKvBadPage);
    return bad | unseen ? -1 : page;
  };
  // The lane's sources: 16 bytes of a code row block, and its place among the
  // scales and biases (keys' scales, biases, values' scales, biases).
  constexpr int kSbChunks = St::kSb / 16;  // 16-byte chunks of one array's tile
  constexpr int kSbIters = (4 * kSbChunks + 31) / 32;
  auto sb_of = [&](int x) -> const uint8_t* {
    const int arr = x / kSbChunks;
    const uint16_t* p = arr == 0 ? a.kv.scales[0] : arr == 1 ? a.kv.biases[0] : arr == 2 ? a.kv.scales[1] : a.kv.biases[1];
    return reinterpret_cast<const uint8_t*>(p) + x % kSbChunks * 16;
  };
  const uint8_t* kc0 = reinterpret_cast<const uint8_t*>(a.kv.codes[0]) + lane * 16;
  const uint8_t* vc0 = reinterpret_cast<const uint8_t*>(a.kv.codes[1]) + lane * 16;
  const uint8_t* sb0 = sb_of(lane % (4 * kSbChunks));
  const uint32_t sb_dst = (lane / kSbChunks >> 1) * St::kHalf + St::kCodes + (lane / kSbChunks & 1) * St::kSb + lane % kSbChunks * 16;
  const int page_mask = (1 << a.kv.page_bits) - 1;
  // Copies keys [16 h0, 16 h1) of a tile whose first key is cache row `row`.
  auto copy = [&](uint32_t dst, long long row, int h0, int h1) {
    constexpr int kHalfCodes = St::kCodes / 2;
    const uint8_t* kc = kc0 + row * (DIM / 2);
    const uint8_t* vc = vc0 + row * (DIM / 2);
#pragma unroll
    for (int i = 0; i < 2 * kHalfCodes; i += 512)
      if (i >= h0 * kHalfCodes && i < h1 * kHalfCodes) {
        cp_async16(dst + lane * 16 + i, kc + i);
        cp_async16(dst + lane * 16 + St::kHalf + i, vc + i);
      }
#pragma unroll
    for (int i = 0; i < kSbIters; ++i) {
      const int x = lane + 32 * i, h = x % kSbChunks >= kSbChunks / 2;  // the half of the tile that the chunk is of
      if (x < 4 * kSbChunks && h >= h0 && h < h1) {
        if (kSbIters == 1)
          cp_async16(dst + sb_dst, sb0 + row * (DIM / 32));
        else
          cp_async16(dst + (x / kSbChunks >> 1) * St::kHalf + St::kCodes + (x / kSbChunks & 1) * St::kSb + x % kSbChunks * 16,
                     sb_of(x) + row * (DIM / 32));
      }
    }
  };
  // Issues tile t into stage s with the pages of its halves; returns which
  // halves are there. One commit group per call, empty or not.
  auto issue = [&](int t, int s, int p0, int p1) -> unsigned {
    const uint32_t dst = ring_s + s * St::kBytes;
    const int in_page = gr.tiles.key0(t) & page_mask;
    auto row_of = [&](int page) { return (((long long)page * a.kv.kv_heads + kvh) << a.kv.page_bits) + in_page; };
    if ((p0 >= 0) & (p1 >= 0) & (page_mask >= kTile - 1)) {
      copy(dst, row_of(p0), 0, 2);
    } else {  // (pages of 16: the second half's page begins where the tile's row 16 is)
      if (p0 >= 0) copy(dst, row_of(p0), 0, 1);
      if (p1 >= 0) copy(dst, row_of(p1) - (page_mask == 15 ? 16 : 0), 1, 2);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return unsigned(p0 >= 0) | unsigned(p1 >= 0) << 1;
  };
  unsigned there = 0;  // two bits per stage
  int at = 0;          // of the warp's tiles: the next one to issue
  int cur0 = pages_of(0, 0), cur1 = pages_of(0, 1);
  auto issue_next = [&](int s) -> unsigned {
    const int p0 = __shfl_sync(~0u, cur0, at & 31), p1 = __shfl_sync(~0u, cur1, at & 31);
    const unsigned h = issue(t_begin + warp + kWarps * at, s, p0, p1);
    if ((++at & 31) == 0) cur0 = pages_of(at, 0), cur1 = pages_of(at, 1);
    return h;
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) there |= issue_next(s) << (2 * s);

  // Query fragments: the B fragments of steps 2 m and 2 m + 1 hold the eight
  // dims of a word as pairs (0, 4), (1, 5) and (2, 6), (3, 7). The scores are
  // multiplied by |scale|; a negative scale flips the queries, 0 clears them.
  const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
  uint2* qs = reinterpret_cast<uint2*>(smem);
  uint2 qr[C::kQReg ? NT : 1][C::kQReg ? kSteps : 1];
#pragma unroll
  for (int e = 0; e < kQWords; ++e) {
    uint4 v = qw[e];
    if (a.scale == 0.f) v = make_uint4(mul2(v.x, 0), mul2(v.y, 0), mul2(v.z, 0), mul2(v.w, 0));
    const uint2 lo = make_uint2(__byte_perm(v.x, v.z, 0x5410) ^ flip, __byte_perm(v.x, v.z, 0x7632) ^ flip);
    const uint2 hi = make_uint2(__byte_perm(v.y, v.w, 0x5410) ^ flip, __byte_perm(v.y, v.w, 0x7632) ^ flip);
    if (C::kQReg) {
      qr[C::kQReg ? e / KW : 0][C::kQReg ? 2 * (e % KW) : 0] = lo;
      qr[C::kQReg ? e / KW : 0][C::kQReg ? 2 * (e % KW) + 1 : 0] = hi;
    } else {
      const int x = e * kWarps + warp, n = x / KW, m = x % KW;
      qs[(n * kSteps + 2 * m) * 32 + lane] = lo;
      qs[(n * kSteps + 2 * m + 1) * 32 + lane] = hi;
    }
  }
  __syncthreads();

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
  const float to_log2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * (1.4426950408889634f * kUnscale);
  // Key of fragment index i (0..15) in a 16-key half of a tile: the two rows
  // of each pair swap for every other pair, which spreads both the key and
  // the value reads over the shared-memory banks.
  const int krow = 2 * (g >> 1) + ((g & 1) ^ ((g >> 1) & 1));
  const int vrow0 = 2 * c + (c & 1), vrow1 = 2 * c + ((c & 1) ^ 1);
  // byte selector: this lane's group of rows 2 c and 2 c + 1, from the words of the two rows, in the rows' fragment order
  uint32_t vsel;
  {
    const uint32_t odd = DIM == 64 ? 0 : DIM == 128 ? g >> 2 : (g >> 1) & 1;  // second group of its word
    const uint32_t r0 = DIM == 64 ? 0x10 : 0x10 + 0x22 * odd, r1 = DIM == 64 ? 0x32 : 0x54 + 0x22 * odd;
    vsel = c & 1 ? r0 << 8 | r1 : r1 << 8 | r0;
  }

  int stage = 0;
  for (int t = t_begin + warp; t < t_end; t += kWarps) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");  // this lane's copies of the tile
    __syncwarp();                                                          // and the other lanes'
    const unsigned have = (there >> (2 * stage)) & 3u;
    const uint8_t* kc = ring + stage * St::kBytes;
    const uint8_t* vc = kc + St::kHalf;
    const int k0 = gr.tiles.key0(t);
    const bool whole = (have == 3) & (k0 + kTile - 1 <= gr.minpos) &
                       ((a.window == 0) | (k0 > gr.maxpos - a.window) | (k0 + kTile <= a.sinks));

    if (!whole) {  // a slot that no row sees may hold anything: its zero probability needs a finite value
      const int key = k0 + lane;
      const bool used = ((have >> (lane >> 4)) & 1u) && key <= gr.maxpos && (a.window == 0 || key >= lo_all || key < a.sinks);
      if (!used) {
        uint16_t* z = reinterpret_cast<uint16_t*>(ring + stage * St::kBytes + St::kHalf + St::kCodes) + lane * (DIM / 64);
#pragma unroll
        for (int i = 0; i < DIM / 64; ++i) z[i] = z[i + St::kSb / 2] = 0;
      }
      __syncwarp();
    }

    // scores; with one row tile two sums, which halves the chain of dependent products
    constexpr int kTwo = NT == 1 ? 1 : 0;
    float sc[NT][2][4], sc2[1][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][u][i] = sc2[n < kTwo ? n : 0][i] = 0.f;
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
            mma(h && n < kTwo ? sc2[n < kTwo ? n : 0] : sc[n][u], p[0][2 * h], p[1][2 * h], p[0][2 * h + 1], p[1][2 * h + 1],
                C::kQReg ? qr[C::kQReg ? n : 0][C::kQReg ? 2 * j + h : 0] : qs[(n * kSteps + 2 * j + h) * 32 + lane]);
      }
      if (kTwo)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[0][u][i] += sc2[0][i];
    }
    // what a row does not see is -inf
    if (!whole) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int pos = si.kv - si.n_new + f.token(rg * C::kRows + 8 * n + 2 * c + i);
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
    float mx[NT][2];  // of this lane's keys
    bool grew = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[n][i] = fmaxf(fmaxf(sc[n][0][i], sc[n][0][2 + i]), fmaxf(sc[n][1][i], sc[n][1][2 + i])) * to_log2;
        grew |= mx[n][i] > m[n][i] + 8.f;
      }
    if (__any_sync(~0u, grew)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float al[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v = fmaxf(m[n][i], mx[n][i]);
#pragma unroll
          for (int off = 4; off <= 16; off <<= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, off));
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
    // probabilities, rounded to the products' type, bf16, after the sums have taken them in fp32 (outputs 0.0020 to 0.0024
    // off the 64-bit result, relative to its norm, where the output's own rounding makes 0.0017), and transposed to the
    // B fragments of the value product
    uint2 pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float r0 = m[n][0] == -INFINITY ? 0.f : m[n][0], r1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float* s = sc[n][u];
        s[0] = ex2(fmaf(s[0], to_log2, -r0)), s[1] = ex2(fmaf(s[1], to_log2, -r1));
        s[2] = ex2(fmaf(s[2], to_log2, -r0)), s[3] = ex2(fmaf(s[3], to_log2, -r1));
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
      }
      // scales and biases of the key pairs, from neighbouring rows
      Sb sb[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* ps = vc + St::kCodes + (16 * u + 8 * h + 2 * c) * (DIM / 32);
        uint32_t s2, b2;
        if (DIM == 64) {  // one group: two rows are one word
          s2 = __byte_perm(*reinterpret_cast<const uint32_t*>(ps), 0, vsel);
          b2 = __byte_perm(*reinterpret_cast<const uint32_t*>(ps + St::kSb), 0, vsel);
        } else if (DIM == 128) {  // two groups: a word per row
          const uint2 sw = *reinterpret_cast<const uint2*>(ps), bw = *reinterpret_cast<const uint2*>(ps + St::kSb);
          s2 = __byte_perm(sw.x, sw.y, vsel), b2 = __byte_perm(bw.x, bw.y, vsel);
        } else {  // four groups: this lane's is in word g / 4 of the two of a row
          const uint8_t* pg = ps + (g >> 2) * 4;
          s2 = __byte_perm(*reinterpret_cast<const uint32_t*>(pg), *reinterpret_cast<const uint32_t*>(pg + 8), vsel);
          b2 = __byte_perm(*reinterpret_cast<const uint32_t*>(pg + St::kSb), *reinterpret_cast<const uint32_t*>(pg + St::kSb + 8), vsel);
        }
        sb[h] = make_sb(s2, b2);
      }
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
    const unsigned h = issue_next(stage);
    there = (there & ~(3u << (2 * stage))) | h << (2 * stage);
    if (++stage == kStages) stage = 0;
  }

  // Merge of the four warps. Sums over the lanes that share a row first; then
  // every (row tile, value word) of the output has an owner warp, which adds
  // the others' fragments from the ring's place and writes it: a lane holds
  // eight neighbouring dims of two rows.
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
  float4* buf = reinterpret_cast<float4*>(smem + C::kOffRing);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float fac[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * C::kRows + 8 * n + 2 * c + i].x);
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = ml[w * C::kRows + 8 * n + 2 * c + i];
        sum += ex2(v.x - ref) * v.y;
      }
      // kUnscale: the values' 2^-23
      fac[i] = sum != 0.f ? ex2(m[n][i] - ref) / sum * kUnscale : 0.f;
      l[n][i] = sum != 0.f ? top + log2f(sum) : -INFINITY;
    }
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      const int owner = (n * VW + w) % kWarps;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float(&x)[4] = o[n][4 * w + k];
        x[0] *= fac[0], x[1] *= fac[1], x[2] *= fac[0], x[3] *= fac[1];
        if (warp != owner)
          buf[(((n * VW + w) * 3 + warp - (warp > owner)) * 4 + k) * 32 + lane] = make_float4(x[0], x[1], x[2], x[3]);
      }
    }
  }
  __syncthreads();
  const bool cut_item = t_begin > 0 || t_end < sq.tiles.n;
  const int slot = 2 * blockIdx.x + (t_begin > 0);  // a CTA's parts: one that begins in an item, one that ends in one
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      if (warp != (n * VW + w) % kWarps) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int from = 0; from < 3; ++from) {
          const float4 v = buf[(((n * VW + w) * 3 + from) * 4 + k) * 32 + lane];
          float(&x)[4] = o[n][4 * w + k];
          x[0] += v.x, x[1] += v.y, x[2] += v.z, x[3] += v.w;
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * n + 2 * c + i;
        if (row >= gr.n_rows) continue;
        const int r = rg * C::kRows + row, t = f.token(r), d = 8 * (VW * g + w);
        const long long at = (long long)(si.first + t) * a.heads + kvh * a.group + r - t * a.group;
        float v[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[2 * k] = o[n][4 * w + k][i], v[2 * k + 1] = o[n][4 * w + k][2 + i];
        if (!cut_item) {
          uint32_t h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[k]) : "f"(v[2 * k + 1]), "f"(v[2 * k]));
          *reinterpret_cast<uint4*>(a.out + at * DIM + d) = make_uint4(h[0], h[1], h[2], h[3]);
          if (g == 0 && w == 0 && a.lse) a.lse[at] = l[n][i] * 0.6931471805599453f;
        } else {
          float4* dst = reinterpret_cast<float4*>(f.part_o + (size_t(slot) * C::kRows + row) * DIM + d);
          dst[0] = make_float4(v[0], v[1], v[2], v[3]);
          dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          if (g == 0 && w == 0) f.part_lse[slot * C::kRows + row] = l[n][i];
        }
      }
    }
  ++item;
  __syncthreads();  // the merge's place becomes the ring's again
  }
  // Launched beside the many-row kernels it has not waited for them: it does not end before them, so that what
  // follows on the stream may rely on both.
  griddep_wait();
}

// Where an item's parts are: parts p = 0 .. n - 1 of CTAs p0 + p. Part 0 ends
// its CTA's range and is in slot 0; the others begin theirs inside the item,
// in slot 1. Items that are not cut have nothing to join, and short sequences
// under a large bound may leave none that is: the combine kernels' threads
// wait for the kernel before on every way out, or their grid could end before
// the one that writes the output, with only the combine for what follows on
// the stream to be ordered behind.
struct Parts {
  SeqItems sq;
  int kvh, rg, n_rows, p0, n;
  __device__ __forceinline__ int slot(int p) const { return 2 * (p0 + p) + (p > 0); }
  // place of row `row` of the group in the outputs
  __device__ __forceinline__ long long place(const FewArgs& f, int rows_per_group, int row) const {
    const int r = rg * rows_per_group + row, t = f.token(r);
    return (long long)(sq.s.first + t) * f.a.heads + kvh * f.a.group + r - t * f.a.group;
  }
};
// The parts of item x of the grid's items (by one CTA of 256 threads; what
// they are counted from is input, so this runs beside the kernel before).
__device__ __forceinline__ Parts parts_of(const FewArgs& f, int x, int rows_per_group) {
  __shared__ long long sums[256];
  Parts q;
  q.n = 0;
  const int per_seq = f.a.kv.kv_heads * f.row_groups;
  const int b = x / per_seq, y = x - b * per_seq;
  q.kvh = y / f.row_groups;
  q.rg = y - q.kvh * f.row_groups;
  q.sq = items_of(f, b, rows_per_group);
  q.n_rows = min(q.sq.rows - q.rg * rows_per_group, rows_per_group);
  if (q.n_rows <= 0) return q;
  // the units of the sequences before, then of the items before
  Cut<256> cut(f, rows_per_group, sums);
  long long u0 = 0;
  for (int c0 = 0; c0 <= b && f.a.kv.n_seqs > 1; c0 += 256) {
    const long long n = f.a.kv.n_seqs <= 256 ? cut.total : cut.chunk(c0);
    u0 += b < c0 + 256 ? (b > c0 ? sums[b - c0 - 1] : 0) : n;
  }
  u0 += (long long)(q.kvh * q.sq.groups + q.rg) * (kItemCost + q.sq.tiles.n) + kItemCost;  // its first tile
  q.p0 = cut.cta_of(u0);
  q.n = cut.cta_of(u0 + q.sq.tiles.n - 1) - q.p0 + 1;
  return q;
}

// Joins the parts of the items that are cut: out = sum_p 2^(lse_p - max) o_p /
// sum_p 2^(lse_p - max). A warp per row, a CTA per eight rows of an item; the
// lanes first hold the parts' weights, then the dims, with eight parts' loads
// in flight, the first eight while the weights are made: bound by this chain of
// loads. (16 sequences of 4 tokens, 13 parts an item: the call 24.7 us, 26.3
// with the weights first; the same for few items below gains nothing.)
template <int DIM>
__global__ void __launch_bounds__(256) attention_combine_kernel(const FewArgs f, int rows_per_group) {
  constexpr int kV = DIM / 128 + (DIM < 128);  // float4 of a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.y * 8 + warp;
  const Parts q = parts_of(f, blockIdx.x, rows_per_group);
  if (q.n <= 1 || row >= q.n_rows) return griddep_wait();  // (see Parts)
  const long long at = q.place(f, rows_per_group, row);
  griddep_wait();
  const bool mine = DIM >= 128 || lane < DIM / 4;
  float4 v[8][kV];
  auto load = [&](int p) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < kV; ++k)
        v[i][k] = mine && p + i < q.n ? reinterpret_cast<const float4*>(
                                            f.part_o + (size_t(q.slot(p + i)) * rows_per_group + row) * DIM)[lane + 32 * k]
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  load(0);  // on their way while the weights are made
  float top = -INFINITY;
  for (int p = lane; p < q.n; p += 32) top = fmaxf(top, f.part_lse[q.slot(p) * rows_per_group + row]);
#pragma unroll
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, off));
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  float4 o[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = 0; c0 < q.n; c0 += 32) {
    const int n = min(32, q.n - c0);
    const float w = lane < n ? ex2(f.part_lse[q.slot(c0 + lane) * rows_per_group + row] - ref) : 0.f;
    for (int p = 0; p < n; p += 8) {
      if (c0 + p) load(c0 + p);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float wi = __shfl_sync(~0u, w, p + i);
        sum += wi;
#pragma unroll
        for (int k = 0; k < kV; ++k)
          o[k].x += wi * v[i][k].x, o[k].y += wi * v[i][k].y, o[k].z += wi * v[i][k].z, o[k].w += wi * v[i][k].w;
      }
    }
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  if (mine)
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      uint2 h;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h.x) : "f"(o[k].y * inv), "f"(o[k].x * inv));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h.y) : "f"(o[k].w * inv), "f"(o[k].z * inv));
      *reinterpret_cast<uint2*>(f.a.out + at * DIM + 4 * (lane + 32 * k)) = h;
    }
  if (lane == 0 && f.a.lse) f.a.lse[at] = sum != 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// The same for few items with many parts each, which want all of the GPU: a
// CTA per (item, row, 64 dims), sixteen threads on the dims and sixteen such
// groups on the parts, eight loads in flight each.
template <int DIM>
__global__ void __launch_bounds__(256) attention_combine_wide_kernel(const FewArgs f, int rows_per_group, int rows) {
  constexpr int kLanes = 16, kGroups = 16;
  constexpr int kMaxParts = 1024;  // (no item has more parts than there are CTAs)
  __shared__ float weight[kMaxParts];
  __shared__ float4 acc[kGroups][kLanes];
  __shared__ float red[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.x % rows;
  const Parts q = parts_of(f, blockIdx.x / rows, rows_per_group);
  const int n = q.n;
  if (n <= 1 || row >= q.n_rows) return griddep_wait();  // (see Parts)
  const long long at = q.place(f, rows_per_group, row);
  const int grp = threadIdx.x / kLanes, d = blockIdx.y * 64 + 4 * (threadIdx.x % kLanes);
  griddep_wait();
  float top = -INFINITY;
  for (int p = threadIdx.x; p < n; p += 256) {
    const float v = f.part_lse[q.slot(p) * rows_per_group + row];
    weight[p] = v;
    top = fmaxf(top, v);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, off));
  if (lane == 0) red[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) top = fmaxf(top, red[w]);
  const float ref = top == -INFINITY ? 0.f : top;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int p1 = grp; p1 < n; p1 += 8 * kGroups) {
    float4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int p = p1 + k * kGroups;
      v[k] = p < n ? *reinterpret_cast<const float4*>(f.part_o + (size_t(q.slot(p)) * rows_per_group + row) * DIM + d)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int p = p1 + k * kGroups;
      const float w = p < n ? ex2(weight[p] - ref) : 0.f;
      sum += w;
      o.x += w * v[k].x, o.y += w * v[k].y, o.z += w * v[k].z, o.w += w * v[k].w;
    }
  }
  acc[grp][threadIdx.x % kLanes] = o;
  __syncthreads();  // (and everyone has read the maxima)
  if (threadIdx.x % kLanes == 0) red[grp] = sum;
  __syncthreads();
  if (grp == 0) {
    float tot = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const float4 w = acc[k][threadIdx.x];
      tot += red[k];
      v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
    const float inv = tot != 0.f ? 1.f / tot : 0.f;
    uint2 h;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h.x) : "f"(v.y * inv), "f"(v.x * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h.y) : "f"(v.w * inv), "f"(v.z * inv));
    *reinterpret_cast<uint2*>(f.a.out + at * DIM + d) = h;
    if (d == 0 && f.a.lse) f.a.lse[at] = tot != 0.f ? (top + log2f(tot)) * 0.6931471805599453f : -INFINITY;
  }
}

// Host plan: row tiles per group (from the most rows a sequence can have),
// and whether items are cut.
struct FewPlan {
  int nt, row_groups, whole, ctas;
  size_t part_rows;
};

FewPlan plan(const AttnArgs& a, int max_rows) {
  FewPlan p;
  const long long rows = std::min<long long>((long long)a.kv.max_new * a.group, max_rows);
  p.nt = rows <= 8 ? 1 : rows <= 16 || a.kv.dim == 256 ? 2 : 4;
  p.row_groups = std::max(1, int((rows + 8 * p.nt - 1) / (8 * p.nt)));
  long long keys = a.kv.max_kv;
  const long long tokens = std::min<long long>(a.kv.max_new, max_rows / a.group + 1);  // of a sequence taken here
  if (a.window > 0)
    keys = std::min<long long>(keys, (long long)a.window + std::min(a.sinks, a.kv.max_kv) + tokens + 2 * kTile);
  p.whole = keys <= whole_keys(a.kv.dim, 1ll * p.row_groups * a.kv.kv_heads * a.kv.n_seqs);
  const int per_sm = a.kv.dim * p.nt <= 128 ? 4 : 2;  // CTAs that fit (registers and the rings)
  p.ctas = num_sms() * per_sm;
  p.part_rows = size_t(2) * p.ctas * 8 * p.nt;  // (there for whole items, too: fewer of them may be cut)
  return p;
}

template <int DIM, int NT>
cudaError_t launch(const FewArgs& f, bool beside, const KvCall& c) {
  using C = FewCfg<DIM, NT>;
  const void* fn = reinterpret_cast<const void*>(&attention_few_kernel<DIM, NT>);
  if (!ensure_smem_limit(fn, C::kSmem)) return cudaErrorInvalidValue;
  const long long items = 1ll * f.row_groups * f.a.kv.kv_heads * f.a.kv.n_seqs;
  // 32 bits number the items' rows and a sequence's units. (The choice by sizes stays far below, with at most 2^30 of the
  // latter; with this kernel asked for, a prompt of 2^15 tokens over 2^20 keys may not.)
  const long long units = 1ll * f.row_groups * f.a.kv.kv_heads * (kItemCost + f.a.kv.max_kv / kTile + 2);
  if (items * C::kRows > 0x7fffffff || units > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(f.whole ? items : f.max_ctas));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = beside ? 1 : 0;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, attention_few_kernel<DIM, NT>, f)) return e;
  if (cudaError_t e = c.launched("attention_few")) return e;
  if (f.whole) return cudaSuccess;
  const int rows = int(std::min<long long>({(long long)f.a.kv.max_new * f.a.group, f.max_rows, C::kRows}));
  const bool wide = items * 32 <= f.max_ctas;  // more than 32 parts each
  cfg = {};
  cfg.gridDim = wide ? dim3(unsigned(items * rows), DIM / 64) : dim3(unsigned(items), (rows + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaError_t e = wide ? cudaLaunchKernelEx(&cfg, attention_combine_wide_kernel<DIM>, f, C::kRows, rows)
                           : cudaLaunchKernelEx(&cfg, attention_combine_kernel<DIM>, f, C::kRows))
    return e;
  return c.launched("attention_combine");
}

}  // namespace

size_t attention_few_workspace(const AttnArgs& a, int max_rows) {
  const FewPlan p = plan(a, max_rows);
  return p.part_rows * (size_t(a.kv.dim) + 1) * 4;
}

long long attention_few_items(const AttnArgs& a, int max_rows) {
  return 1ll * plan(a, max_rows).row_groups * a.kv.kv_heads * a.kv.n_seqs;
}

cudaError_t attention_few(const AttnArgs& a, int max_rows, void* ws, bool beside, const KvCall& c) {
  const FewPlan p = plan(a, max_rows);
  float* part = static_cast<float*>(ws);
  const FewArgs f{a,    max_rows, p.row_groups, p.whole, p.ctas, part, part + p.part_rows * a.kv.dim,
                  ((1ull << 32) + a.group - 1) / a.group};
  switch (a.kv.dim * 8 + p.nt) {
    case 64 * 8 + 1: return launch<64, 1>(f, beside, c);
    case 64 * 8 + 2: return launch<64, 2>(f, beside, c);
    case 64 * 8 + 4: return launch<64, 4>(f, beside, c);
    case 128 * 8 + 1: return launch<128, 1>(f, beside, c);
    case 128 * 8 + 2: return launch<128, 2>(f, beside, c);
    case 128 * 8 + 4: return launch<128, 4>(f, beside, c);
    case 256 * 8 + 1: return launch<256, 1>(f, beside, c);
    default: return launch<256, 2>(f, beside, c);
  }
}

}  // namespace moe
