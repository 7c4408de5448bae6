// Attention of many rows (prompts and chunks) over the 4-bit cache, on the
// tcgen05 tensor cores.
//
// Two matrix products per (row, key): 4 DIM operations, and a cached element
// is used by every row of its kv head, so the products bound the work. The
// codes are therefore expanded once per call, not once per row tile:
//
//   expand   writes the visible keys and values as bf16 tiles of 128 keys into
//            the workspace, laid out exactly as the MMA reads shared memory
//            (128-byte-swizzled, keys K-major; values transposed, so K-major
//            in the second product too), each tile as the halves that the two
//            CTAs of a pair keep. It stays in L2.
//            One extra CTA cuts the work (below).
//   many     S = Q K^T per 128-row tile and 128 keys into tensor memory, the
//            softmax warps turn it into P (bf16, there too), O += P V with
//            P read from tensor memory.
//            The CTA that finishes a row tile's last part joins the parts, if
//            there are few; many parts of few row tiles are joined by
//   combine  over all of the GPU.
//
// The cut: a unit is one row tile times one key tile. All units of all
// sequences and kv heads are numbered row tile by row tile, and each of the CTA
// pairs, one per two SMs, takes an equal, contiguous range, so that neither
// causal masks, ragged lengths nor few row tiles leave SMs idle. A row tile that
// falls into several ranges leaves fp32 partial outputs.
//
// Two CTAs on neighbouring SMs work as one (cta_group::2): an MMA takes 128
// rows of each and all of a key tile, of which each SM keeps half (64 keys, or
// half of the values' dims). A single CTA with the whole key tile is bound by
// its shared memory: per S tile of 128 rows, 128 keys and 128 dims it reads 64
// KB for S and 32 KB for O and takes in 32 KB, 1024 cycles at 128 bytes, as
// long as the products themselves; together they took 1400. The pair reads and
// takes in 40 KB less.
//
// A CTA holds QT row tiles of 128 (two for heads of 64, else one). S tiles
// alternate between two slots in tensor memory.
//   Heads of 64 and 128: P has a place of its own beside S. S(x + 2) is issued
//   as soon as S(x) has been read, and the softmax's two warpgroups work on two
//   S tiles at a time, a thread per row: of two row tiles (64), or the same row
//   tile's in turn (128), with the row's reference maximum handed on.
//   Heads of 256: the output leaves room for two S slots alone, and P takes its
//   S's place: S(0) S(1) | P(0) V, S(2) | P(1) V, S(3) | ... Both warpgroups
//   take half of the keys of every S tile, which halves the time between S and
//   P, in which the slot's products wait.
// The pair's first CTA issues the MMAs; the other tells it which of its
// operands have landed.
//
// Measured: 1024 tokens at 32K positions, 16 heads over 2 of 256 dims, 288 us (307
// once the power limit holds the clock down) with the 20 of the expansion, 541
// GFLOP, 1.9 PFLOP/s in 277 us of the kernel alone: the tensor
// cores are busy in 89% of its cycles. A prompt of 4096, 16 heads over 2 of 128
// dims: 72 us, 69 GFLOP; of that the start and four outputs per pair are about a
// third (between a segment's last P and the next one's first nothing is
// multiplied), the rest is bound by the warp that issues the products, at about
// 1600 cycles per S tile and its product where the tensor cores need 1024.
// Windowed prompts with heads of 64 (three of 1100 to 4001 tokens, window 512): 56
// us, and no unit is busy: the exponentials' pipe 19% of the active cycles, the
// ALU 30%, issue slots 36%, tensor cores 19%. A row tile of 512 rows meets six key tiles
// and the sinks', and every S tile's chain of product, softmax and hand-over stands
// in line, as do each segment's set-up and output; SMs are active in 79% of the time.
//
// Probabilities meet the values as bf16: the products take both operands in one
// type, and the values are bf16. Each is rounded by 2^-9 at most, after the sum
// has taken it in fp32: outputs 0.0021 to 0.0024 off the 64-bit result, relative
// to its norm, where fp32 probabilities and the output's own rounding make 0.0017.
#include <algorithm>

#include "kv.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kBK = 128;                  // keys per tile
constexpr uint32_t kQBlock = 16384;       // 128 query rows of 64 dims
constexpr int kSoftWarps = 8, kWarpTma = 8, kWarpMma = 9, kWarpLoad = 10, kLoadWarps = 2, kThreads = 384;
constexpr int kDescs = 4;                 // segment descriptors in flight
constexpr int kMinUnits = 4;              // of a pair. (16 heads over 2 of 128 dims, one sequence, 64 tokens: over 8000
                                          // keys 25.2 us, with at least 2 units 25.8, 8 units 26.6; over 1000 keys 19.3,
                                          // 18.7, 22.9.)
constexpr int kTileCost = 3;              // units added to every row tile: its set-up and output. (A prompt of 4096 with
                                          // heads of 128: 76 us, with 2 units 79, 5 units 76, 8 units 80.)

template <int DIM>
struct ManyCfg {
  static constexpr int QT = DIM == 64 ? 2 : 1;
  static constexpr int kRows = 128 * QT;  // of a CTA
  static constexpr int kPairRows = 2 * kRows;
  static constexpr int UN = DIM / 64;     // blocks of 64 dims
  static constexpr uint32_t kSlot = 128u * DIM;  // half a key or value tile: what one CTA of the pair keeps
  static constexpr uint32_t kTileBytes = 2 * kSlot;
  static constexpr int kRing = DIM == 64 ? 12 : DIM == 128 ? 11 : 4;
  static constexpr uint32_t kQTile = 128 * DIM * 2;
  static constexpr bool kOwnP = DIM <= 128;    // P has tensor memory of its own; else it takes S's place
  // The softmax's two warpgroups take: DIM 64 a row tile each; 128 S tiles in turn; 256 half of the keys of each S tile.
  static constexpr bool kTurns = DIM == 128, kHalves = DIM == 256;
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffRing = QT * kQTile;
  static constexpr uint32_t kOffEx = kOffRing + kRing * kSlot;  // [2][2][128] floats: exchanged between the warpgroups; [128]: reference maxima
  static constexpr uint32_t kOffBar = kOffEx + (2 * 2 + 1) * 128 * 4;
  // full, empty [kRing]; qfull, qempty, ofree, drain, pq; sfull, pready, sread [2]; pvdone [4]; dfull, dempty, info [kDescs]
  static constexpr int kBars = 2 * kRing + 5 + 10 + 3 * kDescs;
  static constexpr uint32_t kOffDesc = (kOffBar + kBars * 8 + 15) & ~15u;
  static constexpr uint32_t kOffInfo = kOffDesc + kDescs * 80;
  static constexpr uint32_t kOffMisc = kOffInfo + kDescs * 16;
  static constexpr uint32_t kSmem = kOffMisc + 16 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

struct __align__(16) RowTile {
  int seq, row0;        // sequence, first row within it
  int first, n_new, kv;  // of the sequence
  int pad[3];
  __device__ __forceinline__ SeqInfo info() const { return SeqInfo{first, n_new, kv}; }
};

struct PlanHdr {
  long long units;  // of one kv head
  int row_tiles, pad;
};

struct __align__(16) PairRange {
  long long begin;  // first unit of all kv heads' units
  int head, rt;     // its kv head and row tile
};

struct ManyArgs {
  AttnArgs a;
  int max_few;             // sequences with at most this many rows are not taken
  int b0, nb, h0, nh;      // sequences and kv heads of this pass
  int tiles_max;           // key tiles per (sequence, kv head) in the expanded arrays
  uint8_t* kx;             // expanded keys, values: [nb][nh][tiles_max] tiles
  uint8_t* vx;
  uint8_t* bad;            // [nb][tiles_max]: bit i set if the page of keys 16 i .. 16 i + 15 is missing
  PlanHdr* plan;
  long long* unit_off;     // [row tiles + 1] first unit of each row tile (kTileCost + its key tiles each)
  RowTile* row_tile;
  PairRange* range;        // [pairs + 1] where each pair's units begin; the last entry ends them
  int max_row_tiles;
  int pairs;               // CTA pairs of the many kernel
  int* arrived;            // [pairs][2] parts written of the row tile whose first part is the pair's, per CTA
  bool join;               // the kernel joins the parts (else the combine kernel does)
  float* part_o;           // [2 pairs][2][rows][DIM]: two slots per pair, each CTA's rows
  float* part_lse;         // [2 pairs][2][rows], base 2
  unsigned long long inv_group;  // ceil(2^32 / group): row / group for rows below 2^26
  __device__ __forceinline__ int token(int row) const { return int((unsigned(row) * inv_group) >> 32); }
};

// Key tiles that rows at positions minpos .. maxpos read: sink tiles [0,
// n_sink), then [first, first + n - n_sink); at least one, so that rows that
// see nothing are written too.
struct Range {
  int n_sink, first, n;
  __device__ __forceinline__ int tile(int t) const { return t < n_sink ? t : first + t - n_sink; }
};
__device__ __forceinline__ Range range_of(int minpos, int maxpos, int window, int sinks) {
  Range r{0, 0, 1};
  if (maxpos < 0) return r;
  if (window > 0) {
    r.first = max(0, minpos - window + 1) / kBK;
    r.n_sink = min((min(sinks, maxpos + 1) + kBK - 1) / kBK, r.first);
  }
  r.n = r.n_sink + maxpos / kBK - r.first + 1;
  return r;
}

__device__ __forceinline__ bool taken(const ManyArgs& m, const SeqInfo& s) { return s.n_new * m.a.group > m.max_few; }

__device__ __forceinline__ Range seq_range(const ManyArgs& m, const SeqInfo& s) {
  return range_of(s.kv - s.n_new, s.kv - 1, m.a.window, m.a.sinks);
}
__device__ __forceinline__ Range rows_range(const ManyArgs& m, const SeqInfo& s, int row0, int rows) {
  const int base = s.kv - s.n_new, last = min(row0 + rows, s.n_new * m.a.group) - 1;
  return range_of(base + m.token(row0), base + m.token(last), m.a.window, m.a.sinks);
}

// Byte offset of 16-byte chunk c of row r in a 1024-aligned 128-byte-swizzled K-major block.
__device__ __forceinline__ uint32_t sw128(int r, int c) {
  return uint32_t((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}

// ---- the cut ------------------------------------------------------------------------------

constexpr int kPlanThreads = 256;

// Inclusive scan over the CTA of one value per thread; *total gets the sum.
__device__ long long block_scan(long long v, long long* total, long long* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long u = __shfl_up_sync(~0u, v, off);
    if (lane >= off) v += u;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = v;
  __syncthreads();
  long long before = 0, sum = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += buf[w];
    sum += buf[w];
  }
  *total = sum;
  return v + before;
}

__device__ void make_plan(const ManyArgs& m, int rows) {
  __shared__ long long buf[kPlanThreads / 32];
  __shared__ SeqInfo info[kPlanThreads];
  __shared__ int ends[kPlanThreads];  // row tiles up to and with each sequence of the chunk
  long long n_rt = 0, units = 0;
  for (int base = 0; base < m.nb; base += kPlanThreads) {
    const int b = base + threadIdx.x;
    int mine = 0;
    SeqInfo s{0, 0, 0};
    if (b < m.nb) {
      s = kv_seq(m.a.kv, m.b0 + b);
      if (taken(m, s)) mine = (s.n_new * m.a.group + rows - 1) / rows;
    }
    long long total;
    ends[threadIdx.x] = int(block_scan(mine, &total, buf));
    info[threadIdx.x] = s;
    __syncthreads();
    for (int c0 = 0; c0 < total; c0 += kPlanThreads) {
      const int i = c0 + threadIdx.x;
      int n = 0;
      if (i < total && n_rt + i < m.max_row_tiles) {  // (the host's bound; passed only by inconsistent offsets)
        int lo = 0, hi = kPlanThreads - 1;  // the first sequence with ends > i
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (ends[mid] > i)
            hi = mid;
          else
            lo = mid + 1;
        }
        const SeqInfo q = info[lo];
        const int row0 = (i - (lo ? ends[lo - 1] : 0)) * rows;
        m.row_tile[n_rt + i] = RowTile{m.b0 + base + lo, row0, q.first, q.n_new, q.kv, {}};
        n = kTileCost + rows_range(m, q, row0, rows).n;
      }
      long long sum;
      const long long end = block_scan(n, &sum, buf);
      if (n) m.unit_off[n_rt + i] = units + end - n;
      units += sum;
    }
    n_rt += total;
    __syncthreads();
  }
  if (n_rt > m.max_row_tiles) n_rt = m.max_row_tiles;
  if (threadIdx.x == 0) {
    m.unit_off[n_rt] = units;
    m.plan->units = units;
    m.plan->row_tiles = int(n_rt);
  }
  __syncthreads();
  // Pairs that get units: none fewer than kMinUnits, unless there are fewer in all.
  const long long all = units * m.nh, used = max(1ll, min((long long)m.pairs, all / kMinUnits));
  for (int c = threadIdx.x; c <= m.pairs; c += kPlanThreads) {
    const long long begin = all * min((long long)c, used) / used;
    PairRange r{begin, 0, 0};
    if (begin < all) {
      r.head = int(begin / units);
      const long long at = begin - r.head * units;
      int hi = int(n_rt) - 1;  // the last row tile that starts at or before `at`
      while (r.rt < hi) {
        const int mid = (r.rt + hi + 1) >> 1;
        if (m.unit_off[mid] <= at)
          r.rt = mid;
        else
          hi = mid - 1;
      }
    }
    m.range[c] = r;
    if (c < m.pairs) m.arrived[2 * c] = m.arrived[2 * c + 1] = 0;
  }
}

// ---- expand -------------------------------------------------------------------------------

// Pairs (codes in bits 0..3 of both halves of p) -> bf16 scale * code + bias, rounded once.
__device__ __forceinline__ uint32_t dq_pair(uint32_t p, __nv_bfloat162 s2, __nv_bfloat162 b2) {
  const __nv_bfloat162 k128 = __halves2bfloat162(__ushort_as_bfloat16(0x4300), __ushort_as_bfloat16(0x4300));
  const uint32_t x = (p & 0x000F000Fu) | 0x43004300u;
  const __nv_bfloat162 r = __hfma2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), k128), s2, b2);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// CTA 0 makes the plan; the others expand the keys or the values of one key
// tile of one (sequence, kv head): the keys row by row, the values eight keys of eight dims at a time,
// which leaves the transposed 16-byte chunks in registers.
template <int DIM>
__global__ void __launch_bounds__(kPlanThreads) attention_expand_kernel(const ManyArgs m) {
  griddep_launch();
  if (blockIdx.x == 0) {
    make_plan(m, ManyCfg<DIM>::kPairRows);
    return;
  }
  __shared__ long long rows16[kBK / 16];  // first cache row of each 16 keys, -1: zeros
  int x = (blockIdx.x - 1) >> 1;
  const bool values = (blockIdx.x - 1) & 1;
  const int t = x % m.tiles_max;
  x /= m.tiles_max;
  const int h = x % m.nh, bi = x / m.nh, b = m.b0 + bi;
  const KvArgs& kv = m.a.kv;
  const SeqInfo s = kv_seq(kv, b);
  if (!taken(m, s)) return;
  const Range r = seq_range(m, s);
  if (t >= r.n) return;
  const int k0 = r.tile(t) * kBK, minpos = s.kv - s.n_new, maxpos = s.kv - 1;
  const int lo = m.a.window > 0 ? max(0, minpos - m.a.window + 1) : 0;
  if (threadIdx.x < 32) {
    bool missing = false;
    if (threadIdx.x < kBK / 16) {
      const int k = k0 + 16 * threadIdx.x;
      long long row = -1;
      if (k <= maxpos && (k + 16 > lo || k < m.a.sinks)) {
        row = kv_page_row(kv, b, k >> kv.page_bits, m.h0 + h);
        missing = row < 0;
        if (row >= 0) row += k & ((1 << kv.page_bits) - 1);
      }
      rows16[threadIdx.x] = row;
    }
    const unsigned bits = __ballot_sync(~0u, missing);
    if (threadIdx.x == 0 && h == 0 && !values) m.bad[(long long)bi * m.tiles_max + t] = uint8_t(bits);
  }
  __syncthreads();
  const long long tile = ((long long)bi * m.nh + h) * m.tiles_max + t;
  constexpr int W = DIM / 8, G = DIM / 64;
  if (!values) {
    uint8_t* kd = m.kx + tile * ManyCfg<DIM>::kTileBytes;
    // the softmax multiplies by |scale|: a negative scale flips the keys' signs, scale 0 clears them
    const uint32_t flip = m.a.scale < 0.f ? 0x80008000u : 0u, keep = m.a.scale == 0.f ? 0u : 0xFFFFFFFFu;
    constexpr int kBatch = 4;  // loads in flight before the first is used
    static_assert(kBK * W / kPlanThreads % kBatch == 0, "batches of whole passes");
    const int w = threadIdx.x % W;
    for (int p = 0; p < kBK * W / kPlanThreads; p += kBatch) {
      uint32_t c[kBatch];
      uint16_t sc[kBatch], bs[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int key = (p + i) * (kPlanThreads / W) + threadIdx.x / W;
        const long long r16 = rows16[key >> 4];
        c[i] = sc[i] = bs[i] = 0;
        if (r16 >= 0 && k0 + key <= maxpos) {
          const long long row = r16 + (key & 15);
          c[i] = kv.codes[0][row * W + w];
          sc[i] = kv.scales[0][row * G + w / 8];
          bs[i] = kv.biases[0][row * G + w / 8];
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int key = (p + i) * (kPlanThreads / W) + threadIdx.x / W;
        const __nv_bfloat16 s16 = __ushort_as_bfloat16(sc[i]), b16 = __ushort_as_bfloat16(bs[i]);
        uint32_t o[4];
        dq8_bf16(c[i], __halves2bfloat162(s16, s16), __halves2bfloat162(b16, b16), o);
        *reinterpret_cast<uint4*>(kd + (key >> 6) * ManyCfg<DIM>::kSlot + (w / 8) * 8192 + sw128(key & 63, w & 7)) =
            make_uint4((o[0] ^ flip) & keep, (o[1] ^ flip) & keep, (o[2] ^ flip) & keep, (o[3] ^ flip) & keep);
      }
    }
    return;
  }
  uint8_t* vd = m.vx + tile * ManyCfg<DIM>::kTileBytes;
  // lanes: eight 8-key chunks (one 128-byte row of 64 keys) by four words
  for (int e = threadIdx.x; e < (kBK / 8) * W; e += kPlanThreads) {
    const int ko = e & 7, w = (e >> 3) % W, kb = (e >> 3) / W;  // 8-key chunk in its block, word, block of 64 keys
    const int key0 = kb * 64 + ko * 8;
    uint32_t c[8];
    uint32_t sc[8], bs[8];
    const long long r16 = rows16[key0 >> 4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = sc[i] = bs[i] = 0;
      // a slot that no row sees may hold anything: its zero probability needs a finite value
      const int key = k0 + key0 + i;
      if (r16 >= 0 && key <= maxpos && (key >= lo || key < m.a.sinks)) {
        const long long row = r16 + (key0 & 15) + i;
        c[i] = kv.codes[1][row * W + w];
        sc[i] = kv.scales[1][row * G + w / 8];
        bs[i] = kv.biases[1][row * G + w / 8];
      }
    }
    uint32_t o[8][4];  // [dim][pair of keys]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t s2 = sc[2 * i] | sc[2 * i + 1] << 16, b2 = bs[2 * i] | bs[2 * i + 1] << 16;
      const __nv_bfloat162 sp = *reinterpret_cast<const __nv_bfloat162*>(&s2);
      const __nv_bfloat162 bp = *reinterpret_cast<const __nv_bfloat162*>(&b2);
      const uint32_t lo2 = __byte_perm(c[2 * i], c[2 * i + 1], 0x5410), hi2 = __byte_perm(c[2 * i], c[2 * i + 1], 0x7632);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        o[n][i] = dq_pair(lo2 >> (4 * n), sp, bp);
        o[n + 4][i] = dq_pair(hi2 >> (4 * n), sp, bp);
      }
    }
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int d = 8 * w + n;
      constexpr int kHalf = DIM / 2;  // dims of a CTA
      const uint32_t at = d / kHalf * ManyCfg<DIM>::kSlot + kb * (kHalf * 128) + sw128(d % kHalf, ko);
      *reinterpret_cast<uint4*>(vd + at) = make_uint4(o[n][0], o[n][1], o[n][2], o[n][3]);
    }
  }
}

// ---- tcgen05 ------------------------------------------------------------------------------

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups
// 1024 bytes apart, version 1. Low half: the start address in 16-byte units
// and the leading offset; the high half is the same for all.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); }
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << (46 - 32)) | (2u << (61 - 32));
// kind::f16: bf16 A and B, fp32 D, both K-major, M = 256 (128 rows of each CTA of the pair), N = n.
constexpr uint32_t idesc_n(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(256 >> 4) << 24);
}
// Four K = 16 steps of a 64-wide K block, by one elected lane of the converged
// warp: D += A B^T with A in shared memory, or in tensor memory. The first
// step overwrites D when acc is 0. (One asm statement with warp-uniform
// operands: issued by a single lane of a divergent warp, with its operands in
// per-thread registers, an MMA took ~130 cycles to issue, twice its run time.)
__device__ __forceinline__ void umma4_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred e, p, t;\n .reg .b32 x1, x2, x3, y1, y2, y3;\n .reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n"
      " elect.sync _|e, 0xffffffff;\n"
      " add.u32 x1, %1, 2;\n add.u32 x2, %1, 4;\n add.u32 x3, %1, 6;\n"
      " add.u32 y1, %2, 2;\n add.u32 y2, %2, 4;\n add.u32 y3, %2, 6;\n"
      " mov.b64 a0, {%1, %3};\n mov.b64 a1, {x1, %3};\n mov.b64 a2, {x2, %3};\n mov.b64 a3, {x3, %3};\n"
      " mov.b64 b0, {%2, %3};\n mov.b64 b1, {y1, %3};\n mov.b64 b2, {y2, %3};\n mov.b64 b3, {y3, %3};\n"
      " setp.ne.b32 p, %5, 0;\n setp.eq.b32 t, %5, %5;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a0, b0, %4, p;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %4, t;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %4, t;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %4, t;\n}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma4_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred e, p, t;\n .reg .b32 x1, x2, x3, y1, y2, y3;\n .reg .b64 b0, b1, b2, b3;\n"
      " elect.sync _|e, 0xffffffff;\n"
      " add.u32 x1, %1, 8;\n add.u32 x2, %1, 16;\n add.u32 x3, %1, 24;\n"
      " add.u32 y1, %2, 2;\n add.u32 y2, %2, 4;\n add.u32 y3, %2, 6;\n"
      " mov.b64 b0, {%2, %3};\n mov.b64 b1, {y1, %3};\n mov.b64 b2, {y2, %3};\n mov.b64 b3, {y3, %3};\n"
      " setp.ne.b32 p, %5, 0;\n setp.eq.b32 t, %5, %5;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b0, %4, p;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [x1], b1, %4, t;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [x2], b2, %4, t;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [x3], b3, %4, t;\n}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(acc)
      : "memory");
}
// `bar` of both CTAs receives one arrival when every MMA that the elected lane issued before has completed.
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .b16 both;\n elect.sync _|e, 0xffffffff;\n mov.b16 both, 3;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], both;\n}" ::"r"(bar)
      : "memory");
}

// The same for a barrier of this CTA alone.
__device__ __forceinline__ void umma_commit_own(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar)
      : "memory");
}

// Arrives on the first CTA's barrier at this CTA's address `bar`. What it
// tells of is in tensor memory, or came by TMA, and is ordered by the tcgen05
// fences and the copies' own barriers; a release of the whole cluster's memory
// took ~2000 cycles of a softmax warp's time per tile.
__device__ __forceinline__ void arrive_first(uint32_t bar) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(bar));
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}
// The same, with this thread's view of memory released to the first CTA.
__device__ __forceinline__ void arrive_first_release(uint32_t bar) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(bar));
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}
// mbar_wait for such an arrival.
__device__ __forceinline__ bool mbar_wait_acquire(uint32_t bar, uint32_t parity, volatile int* abort_flag, WsHeader* hdr,
                                                  int site) {
  const long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kTrySuspendNs)
        : "memory");
    if (ok) return true;
    if ((i & 15u) == 0) {
      if (*abort_flag) return false;
      if (clock64() - t0 > kWaitLimit) {
        *abort_flag = 1;
        report(hdr, MOE_ERR_DEVICE_TIMEOUT, site);
        return false;
      }
    }
  }
}
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// The wait, with a load's registers as operands: no use of them may be scheduled before it.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 32 bytes, a whole sector, in one store (32-byte aligned).
__device__ __forceinline__ void st_v8(void* dst, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---- the segments of a CTA ------------------------------------------------------------------

// A CTA's rows of a pair's part of a row tile: key tiles [j0, j1) of n. j1 = 0: no more.
struct __align__(16) Segment {
  int seq, head, row0, n_rows;   // sequence and kv head (within the pass), first row, rows
  int j0, j1, n, part;           // part: slot of the partial output, -1 if the row tile is whole
  int first, base_pos, last;     // sequence's first step token, position of its token 0, its last row
  int all_sink, all_first;       // Range of the sequence's expanded tiles
  int my_sink, my_first;         // Range of the row tile
  int pad;
  long long u0;                  // first unit of the row tile
  __device__ __forceinline__ int tile(int j) const { return j < my_sink ? j : my_first + j - my_sink; }
  __device__ __forceinline__ int index(int j) const {
    const int t = tile(j);
    return t < all_first ? t : all_sink + t - all_first;
  }
};
static_assert(sizeof(Segment) == 80, "descriptor size");

// Of a divided row tile: its parts, the first and last pair with units of it.
struct PartInfo {
  int parts, c0, c1, pad;
};

// Key tiles before unit `u` of a row tile of n key tiles that begins at unit u0.
__device__ __forceinline__ int tiles_before(long long u, long long u0, int n) {
  const long long t = u - u0 - kTileCost;
  return t <= 0 ? 0 : t < n ? int(t) : n;
}

// Steps through the units [u, end) of a pair. Every row tile has kTileCost
// units more than key tiles; a part that holds none of the latter is skipped.
struct Cursor {
  const ManyArgs& m;
  long long u, end, units;
  int rt, head;
  const int pair = blockIdx.x >> 1, rank = blockIdx.x & 1;
  __device__ Cursor(const ManyArgs& args) : m(args) {
    const PairRange r = m.range[pair];
    units = m.plan->units;
    u = r.begin;
    end = m.range[pair + 1].begin;
    head = r.head;
    rt = r.rt;
  }
  __device__ void next(Segment* s, int rows) {
    s->j1 = 0;
    while (u < end && s->j1 == 0) {
      const long long base = head * units, o0 = base + m.unit_off[rt], o1 = base + m.unit_off[rt + 1];
      const long long stop = end < o1 ? end : o1;
      const int n = int(o1 - o0) - kTileCost;
      const int j0 = max(0, int(u - o0) - kTileCost), j1 = max(0, int(stop - o0) - kTileCost);
      if (j1 > j0) {
        const RowTile t = m.row_tile[rt];
        const SeqInfo si = t.info();
        const Range all = seq_range(m, si), mine = rows_range(m, si, t.row0, 2 * rows);
        s->seq = t.seq - m.b0;
        s->head = head;
        s->row0 = t.row0 + rank * rows;
        s->last = si.n_new * m.a.group - 1;
        s->n_rows = max(0, min(rows, s->last + 1 - s->row0));
        s->j0 = j0;
        s->j1 = j1;
        s->n = n;
        s->part = j0 == 0 && j1 == n ? -1 : 2 * (2 * pair + (j0 > 0 ? 1 : 0)) + rank;
        s->first = si.first;
        s->base_pos = si.kv - si.n_new;
        s->all_sink = all.n_sink, s->all_first = all.first;
        s->my_sink = mine.n_sink, s->my_first = mine.first;
        s->u0 = o0;
      }
      u = stop;
      if (stop == o1 && ++rt == m.plan->row_tiles) rt = 0, ++head;
    }
  }
};

// (apart from the descriptor: it takes loads that depend on one another, and is needed only at the segment's end)
__device__ __forceinline__ PartInfo part_info(const ManyArgs& m, const Segment& s) {
  const int pair = s.part >> 2;
  PartInfo p{0, pair, pair, 0};
  const long long end = s.u0 + kTileCost + s.n;
  while (m.range[p.c0].begin > s.u0) --p.c0;
  while (m.range[p.c1 + 1].begin < end) ++p.c1;
  for (int c = p.c0, from = 0; c <= p.c1; ++c) {
    const int to = tiles_before(m.range[c + 1].begin, s.u0, s.n);
    p.parts += to > from;
    from = to;
  }
  return p;
}

// Keeps registers that a store to tensor memory may still be reading.
__device__ __forceinline__ void keep(const uint32_t (&p)[32]) {
#pragma unroll
  for (int e = 0; e < 32; e += 8)
    asm volatile("" ::"r"(p[e]), "r"(p[e + 1]), "r"(p[e + 2]), "r"(p[e + 3]), "r"(p[e + 4]), "r"(p[e + 5]), "r"(p[e + 6]),
                 "r"(p[e + 7]));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
// Arrives on `bar` once every cp.async of this thread has landed (counted in the barrier's arrivals).
__device__ __forceinline__ void cp_async_arrive_noinc(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int DIM>
__global__ void __launch_bounds__(kThreads, 1) attention_many_kernel(const ManyArgs m) {
  using C = ManyCfg<DIM>;
  constexpr int QT = C::QT, UN = C::UN, kRing = C::kRing;
  constexpr bool kOwnP = C::kOwnP, kHalves = C::kHalves, kTurns = C::kTurns;
  constexpr int kArrive = kHalves ? kSoftWarps : kSoftWarps / 2;  // softmax warps of an S tile, per CTA
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bar0 = base + C::kOffBar;
  auto full = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty = [&](uint32_t s) { return bar0 + 8u * (kRing + s); };
  const uint32_t qfull = bar0 + 8u * (2 * kRing), qempty = qfull + 8, ofree = qfull + 16, drain = qfull + 24;
  const uint32_t pq = qfull + 32;  // first CTA: the other's queries are there
  auto sfull = [&](uint32_t s) { return qfull + 40 + 8u * s; };
  auto pready = [&](uint32_t s) { return qfull + 56 + 8u * s; };
  auto sread = [&](uint32_t s) { return qfull + 72 + 8u * s; };  // kOwnP: S has been read
  auto pvdone = [&](uint32_t g) { return qfull + 88 + 8u * (g & 3u); };  // of S tile g; phase g / 4
  auto dfull = [&](uint32_t i) { return qfull + 88 + 8u * (4 + i % kDescs); };
  auto dempty = [&](uint32_t i) { return qfull + 88 + 8u * (4 + kDescs + i % kDescs); };
  const bool first_cta = (blockIdx.x & 1) == 0;
  auto info_bar = [&](uint32_t i) { return qfull + 88 + 8u * (4 + 2 * kDescs + i % kDescs); };
  Segment* descs = reinterpret_cast<Segment*>(gbase + C::kOffDesc);
  PartInfo* infos = reinterpret_cast<PartInfo*>(gbase + C::kOffInfo);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::kOffMisc + 4);
  const AttnArgs& a = m.a;
  WsHeader* hdr = a.kv.hdr;
  const int warp = __shfl_sync(~0u, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;  // (known to be warp-uniform)

  if (threadIdx.x == 0) {
    // (the first CTA's slots are full when the other's are, too)
    for (int s = 0; s < kRing; ++s) mbar_init(full(s), first_cta ? 2 : 1), mbar_init(empty(s), 1);
    mbar_init(pq, 1);
    mbar_init(qfull, kLoadWarps * 32);
    mbar_init(qempty, 1);
    mbar_init(ofree, 2 * kSoftWarps);
    for (int i = 0; i < kDescs; ++i) mbar_init(dfull(i), 1), mbar_init(dempty(i), kSoftWarps + 2 + kLoadWarps), mbar_init(info_bar(i), 1);
    for (int s = 0; s < 2; ++s) mbar_init(sfull(s), 1), mbar_init(pready(s), 2 * kArrive), mbar_init(sread(s), 2 * kArrive);
    for (int g = 0; g < 4; ++g) mbar_init(pvdone(g), 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  pair_sync();  // both CTAs' barriers are there
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // S slots at columns 0 and 128, O at 256
  griddep_wait();
  griddep_launch();

  // Ring position of key tile i and value tile i of a segment of n tiles: K0 K1
  // V0 K2 V1 ... (S runs a tile ahead, or two).
  auto k_at = [](int i) { return i == 0 ? 0 : 2 * i - 1; };
  auto v_at = [](int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; };

  // Segment i, once its descriptor is there; every reader arrives on dempty(i) when it needs it no more.
  auto descriptor = [&](uint32_t i, Segment* s, bool& ok) {
    if (ok) ok = mbar_wait(dfull(i), (i / kDescs) & 1u, abort_flag, hdr, kWaitLimit, false, 219);
    s->j1 = 0;
    if (ok) *s = descs[i % kDescs];
    return ok && s->j1 > 0;
  };

  // Registers: launched with 168 per thread; the softmax warps hold a row of S
  // (208), the other four warps need few (88): 2 * 208 + 88 = 3 * 168.
  if (warp >= kSoftWarps) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == kWarpTma) {
    if (lane == 0) {
      Segment s;
      uint32_t it = 0;
      bool ok = true;
      for (uint32_t sg = 0; descriptor(sg, &s, ok); ++sg) {
        mbar_arrive(dempty(sg));
        const long long tile0 = ((long long)s.seq * m.nh + s.head) * m.tiles_max;
        const int n = s.j1 - s.j0;
        for (int p = 0; p < 2 * n && ok; ++p) {
          // which tile has ring position p
          const bool is_v = p == 2 * n - 1 || (p >= 2 && !(p & 1));
          const int i = is_v ? (p == 2 * n - 1 ? n - 1 : p / 2 - 1) : (p + 1) / 2;
          const uint8_t* src = (is_v ? m.vx : m.kx) + (tile0 + s.index(s.j0 + i)) * C::kTileBytes + (first_cta ? 0 : C::kSlot);
          const uint32_t slot = it % kRing;
          if (!(ok = mbar_wait(empty(slot), ((it / kRing) & 1u) ^ 1u, abort_flag, hdr, kWaitLimit, false, 220))) break;
          mbar_arrive_tx(full(slot), C::kSlot);
          bulk_g2s(base + C::kOffRing + slot * C::kSlot, src, C::kSlot, full(slot));
          ++it;
        }
      }
      if (!ok) {  // copies in flight land before the CTA leaves (bounded)
        const uint32_t from = it > kRing ? it - kRing : 0;
        // (the first CTA's barriers may want for the other's arrivals now: one limit is long enough for any copy)
        for (uint32_t i = from; i < it; ++i)
          if (!mbar_wait(full(i % kRing), (i / kRing) & 1u, abort_flag, hdr, kWaitLimit, true, 221)) break;
      }
    }
  } else if (warp == kWarpMma) {
    Segment s;
    bool ok = true;
    uint32_t ring = 0;  // ring slots before this segment
    if (!first_cta) {
      // tells the first CTA what has landed here, in the order in which it needs it
      if (lane == 0) {
        for (uint32_t sg = 0; descriptor(sg, &s, ok); ++sg) {
          mbar_arrive(dempty(sg));
          if (!(ok = mbar_wait(qfull, sg & 1u, abort_flag, hdr, kWaitLimit, false, 233))) break;
          fence_proxy_async();  // the loader warps' copies, for the tensor cores
          arrive_first_release(pq);
          for (int p = 0; p < 2 * (s.j1 - s.j0) && ok; ++p, ++ring) {
            if (!(ok = mbar_wait(full(ring % kRing), (ring / kRing) & 1u, abort_flag, hdr, kWaitLimit, false, 234))) break;
            arrive_first(full(ring % kRing));
          }
        }
      }
    } else {
      // the whole warp, converged; every wait's outcome is made warp-uniform
      uint32_t g0 = 0;  // S tiles before this segment
      auto wait = [&](uint32_t bar, uint32_t parity, int site) {
        ok = __all_sync(~0u, mbar_wait(bar, parity, abort_flag, hdr, kWaitLimit, false, site));
        tc_fence_after();
        return ok;
      };
      constexpr uint32_t kIdS = idesc_n(128), kIdO = idesc_n(DIM);
      for (uint32_t sg = 0;; ++sg) {
        if (!__all_sync(~0u, descriptor(sg, &s, ok))) break;
        if (lane == 0) mbar_arrive(dempty(sg));
        __syncwarp();
        const int n = s.j1 - s.j0, total = n * QT;
        if (!wait(qfull, sg & 1u, 222)) break;
        if (!(ok = __all_sync(~0u, mbar_wait_acquire(pq, sg & 1u, abort_flag, hdr, 235)))) break;
        fence_proxy_async();  // the loader warps' copies, for the tensor core
        auto wait_slot = [&](uint32_t seq) {
          return wait(full(seq % kRing), (seq / kRing) & 1u, 223);
        };
        auto qk = [&](int x) {  // S tile x: row tile x % QT, key tile x / QT
          const int q = x % QT, i = x / QT;
          const uint32_t sl = (g0 + x) & 1u, seq = ring + k_at(i), kb = base + C::kOffRing + seq % kRing * C::kSlot;
          if (q == 0 && !wait_slot(seq)) return;
#pragma unroll
          for (int u = 0; u < UN; ++u)
            umma4_ss(tmem + sl * 128, desc_lo(base + C::kOffQ + q * C::kQTile + u * kQBlock), desc_lo(kb + u * 8192), kIdS, u != 0);
          if (q == QT - 1) umma_commit(empty(seq % kRing));
          umma_commit(sfull(sl));
          if (x == total - 1) umma_commit(qempty);
        };
        auto pv = [&](int x) {  // O of row tile x % QT += P(x) V
          const int q = x % QT, i = x / QT;
          const uint32_t sl = (g0 + x) & 1u, p = kOwnP ? tmem + 384 + sl * 64 : tmem + sl * 128, o = tmem + 256 + q * DIM;
          const uint32_t seq = ring + v_at(i, n), vb = base + C::kOffRing + seq % kRing * C::kSlot;
          if (q == 0 && !wait_slot(seq)) return;
#pragma unroll
          for (int kb = 0; kb < 2; ++kb) umma4_ts(o, p + kb * 32, desc_lo(vb + kb * (DIM * 64)), kIdO, i > 0 || kb > 0);
          if (q == QT - 1) umma_commit(empty(seq % kRing));
          umma_commit(pvdone(g0 + x));
        };
        qk(0);
        if (ok && total > 1) qk(1);
        // kOwnP: once S tile y has been read, S(y + 2) takes its slot. That is before P(y - 1) is there: the warpgroup
        // that reads S(y) has had P(y - 2) behind it.
        auto follow = [&](int y) {
          if (y >= total || !wait(sread((g0 + y) & 1u), ((g0 + y) >> 1) & 1u, 237)) return;
          if (y + 2 < total) qk(y + 2);
        };
        if (kOwnP && ok) follow(0);
        for (int x = 0; x < total && ok; ++x) {
          const uint32_t g = g0 + x;
          if (kOwnP) follow(x + 1);
          if (!ok) break;
          if (!wait(pready(g & 1u), (g >> 1) & 1u, 224)) break;
          if (x == 0 && sg > 0 && !wait(ofree, (sg - 1) & 1u, 230)) break;
          pv(x);
          if (!kOwnP && ok && x + 2 < total) qk(x + 2);
        }
        g0 += total;
        ring += 2 * n;
      }
      // every MMA has completed before the pair leaves (bounded)
      __syncwarp();
      umma_commit_own(drain);
      mbar_wait(drain, 0, abort_flag, hdr, kWaitLimit, true, 225);
    }
  } else {
    // ---------------- segments and query rows: two warps; lane 0 of the first steps through the units ----------
    Cursor cur(m);
    Segment s;
    bool ok = true;
    auto produce = [&](uint32_t i) {
      if (warp != kWarpLoad || lane != 0 || !ok) return;
      if (i >= kDescs && !(ok = mbar_wait(dempty(i), ((i / kDescs) & 1u) ^ 1u, abort_flag, hdr, kWaitLimit, false, 231))) return;
      cur.next(&s, C::kRows);
      descs[i % kDescs] = s;
      mbar_arrive(dfull(i));
    };
    produce(0);
    __syncwarp();
    for (uint32_t sg = 0;; ++sg) {
      if (!__all_sync(~0u, descriptor(sg, &s, ok))) break;
      const Segment mine = s;
      if (sg > 0 && ok) ok = mbar_wait(qempty, (sg - 1) & 1u, abort_flag, hdr, kWaitLimit, false, 232);
      ok = __all_sync(~0u, ok);
      if (!ok) break;
      // A lane looks one row of 32 up, and the warp copies them with the addresses from their lanes: a lookup per chunk
      // made these copies 3 to 4 thousand cycles long, with the segment's first product behind them.
      constexpr int CH = DIM / 8, kStep = 32 / CH;  // 16-byte chunks of a row, rows of one instruction
      const int c = lane % CH, sub = lane / CH;
      const uint16_t* qh = a.q + (m.h0 + mine.head) * a.group * DIM;
      for (int r32 = (warp - kWarpLoad) * 32; r32 < C::kRows; r32 += 32 * kLoadWarps) {
        const int rr = min(mine.row0 + r32 + lane, mine.last), t = m.token(rr);
        const long long src = reinterpret_cast<long long>(qh + (mine.first + t) * a.q_stride + (rr - t * a.group) * DIM);
        const uint32_t dst = base + C::kOffQ + (r32 >> 7) * C::kQTile + (c >> 3) * kQBlock + ((r32 & 127) >> 3) * 1024;
#pragma unroll
        for (int k = 0; k < 32; k += kStep) {
          const long long from = __shfl_sync(~0u, src, k + sub);
          cp_async16(dst + sw128(k + sub, c & 7), reinterpret_cast<const uint16_t*>(from) + c * 8,
                     r32 + k + sub < mine.n_rows ? 16u : 0u);
        }
      }
      cp_async_arrive_noinc(qfull);
      produce(sg + 1);  // the next one, while this one's rows are used
      if (warp == kWarpLoad + 1 && lane == 0) {
        if (mine.part >= 0 && m.join) infos[sg % kDescs] = part_info(m, mine);
        mbar_arrive(info_bar(sg));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(dempty(sg));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---------------- softmax: eight warps ----------------
    // Heads of 64 and 128: a thread has a row of an S tile, and one warpgroup's loads and maxima run beside the other's
    // exponentials. Heads of 64: a row tile each. Heads of 128: the S tiles of one row tile in turn; the reference
    // maximum is the row's, in shared memory, and handed on from tile to tile. Heads of 256: two threads per row with 64
    // keys each, which halves the time between S and P, with the slot's products waiting; they exchange maxima.
    constexpr int kCols = kHalves ? 64 : 128;       // keys of an S tile per thread
    constexpr int kScale = kHalves ? DIM / 2 : DIM;  // dims of O that a thread rescales
    constexpr int kOCols = QT == 1 ? DIM / 2 : DIM;  // dims of O that it writes
    const int wg = warp >> 2, half = kHalves ? wg : 0, ohalf = QT == 1 ? wg : 0, q = QT == 1 ? 0 : wg;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;  // the tensor-memory lanes this warp may access
    float* ex = reinterpret_cast<float*>(gbase + C::kOffEx);
    // |scale| in base 2 (the keys carry the sign; for scale 0 they are zeros)
    const float c2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.4426950408889634f;
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;  // rows are multiples of 128 bytes
    Segment s;
    uint32_t g0 = 0, exn = 0;  // S tiles before this segment, exchanges
    // After a failed wait a warp keeps going without waiting, so that the
    // others never hang in a barrier; the status says that the output is void.
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity, int site) {
      if (ok) ok = mbar_wait(bar, parity, abort_flag, hdr, kWaitLimit, false, site);
    };
    // the other half's value of this row (the two warps that hold it wait for each other)
    auto exchange = [&](float v) {
      float* e = ex + (exn & 1u) * 256;
      ++exn;
      e[wg * 128 + row] = v;
      asm volatile("bar.sync %0, 64;" ::"r"(2 + (warp & 3)) : "memory");
      return e[(wg ^ 1) * 128 + row];
    };
    // kTurns: the rows' reference maxima, read and written between take_turn and pass_turn
    float* refs = ex + 2 * 256;
    auto take_turn = [&] { asm volatile("bar.sync %0, 64;" ::"r"(6 + (warp ^ 4)) : "memory"); };
    auto pass_turn = [&] { asm volatile("bar.arrive %0, 64;" ::"r"(6 + warp) : "memory"); };
    auto wait_product = [&](uint32_t g, int site) { wait(pvdone(g), (g >> 2) & 1u, site); };
    for (uint32_t sg = 0;; ++sg) {
      // The eight warps agree on whether there is a segment: after a failed wait the flag has them all leave here.
      int more = descriptor(sg, &s, ok);
      __syncwarp();
      asm volatile(
          "{\n .reg .pred p;\n setp.ne.b32 p, %0, 0;\n bar.red.and.pred p, 1, %1, p;\n selp.s32 %0, 1, 0, p;\n}"
          : "+r"(more)
          : "n"(kSoftWarps * 32)
          : "memory");
      if (!more) break;
      if (lane == 0) mbar_arrive(dempty(sg));
      float ref = -INFINITY, sum = 0.f;
      const int r0 = s.row0 + q * 128;
      const int pos = s.base_pos + m.token(min(r0 + row, s.last));
      const int minpos = s.base_pos + m.token(min(r0, s.last)), maxpos = s.base_pos + m.token(min(r0 + 127, s.last));
      const int n = s.j1 - s.j0;
      const uint8_t* bad = m.bad + (long long)s.seq * m.tiles_max;
      const int first = kTurns ? (wg ^ g0) & 1 : 0;  // of this warpgroup's tiles
      constexpr int kStep = kTurns ? 2 : 1;
      unsigned bad_next = first < n ? bad[s.index(s.j0 + first)] : 0;
      // S tile g's scores, on their way when this returns
      uint32_t v[kCols];
      auto load = [&](uint32_t g) {
        wait(sfull(g & 1u), (g >> 1) & 1u, 226);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kCols; c += 32) tmem_ld32(tmem + lanes + (g & 1u) * 128 + half * 64 + c, v + c);
      };
      for (int i = first; i < n; i += kStep) {
        const int k0 = s.tile(s.j0 + i) * kBK;
        const unsigned missing = bad_next;
        if (i + kStep < n) bad_next = bad[s.index(s.j0 + i + kStep)];
        const uint32_t g = g0 + i * QT + q, gl = g - QT;  // and the last one before it into the same output
        const uint32_t pl = tmem + lanes + (kOwnP ? 384 + (g & 1u) * 64 : (g & 1u) * 128);
        const uint32_t ocol = tmem + lanes + 256 + q * DIM + half * kScale;
        load(g);
#pragma unroll
        for (int c = 0; c < kCols; c += 32) tmem_wait_ld32(v + c);
        if (kOwnP) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_first(sread(g & 1u));
        }
        const bool whole = missing == 0 && k0 + kBK - 1 <= minpos &&
                           (a.window == 0 || k0 > maxpos - a.window || k0 + kBK <= a.sinks);
        if (!whole) {
#pragma unroll
          for (int c = 0; c < kCols; c += 64) {
            // bit e: this row sees key kb + e, from the interval (or the sinks) that it sees
            const int h = kHalves ? half : c / 64, kb = k0 + h * 64;
            auto below = [](int x) { return x <= 0 ? 0ull : x >= 64 ? ~0ull : (1ull << x) - 1; };  // bits under x
            uint64_t sees = below(pos + 1 - kb);
            if (a.window > 0) sees &= ~below(pos - a.window + 1 - kb) | below(a.sinks - kb);
#pragma unroll
            for (int i16 = 0; i16 < 4; ++i16)
              if ((missing >> (h * 4 + i16)) & 1u) sees &= ~(0xFFFFull << (16 * i16));
            // 32 keys at a time: most of them are seen by every row of the warp
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t bits = uint32_t(sees >> (32 * w));
              if (__all_sync(~0u, bits == ~0u)) continue;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(bits & (1u << e))) v[c + 32 * w + e] = 0xff800000u;  // -inf
            }
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < kCols; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(v[e]));
        float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // the reference maximum moves only when a score passes it by 2^8: probabilities are floating point, so
        // nothing is lost, and the output is hardly ever rescaled
        if (kHalves) top = fmaxf(top, exchange(top));
        if (kTurns) {
          if (g > 0) take_turn();
          const float now = i > 0 ? refs[row] : -INFINITY;
          if (now != ref) sum *= ex2(ref - now), ref = now;
        }
        const bool grew = __any_sync(~0u, top * c2 > ref + 8.f);
        float al = 1.f;
        if (grew) {
          const float to = fmaxf(ref, top * c2);
          al = to == -INFINITY ? 1.f : ex2(ref - to);
          ref = to;
          sum *= al;
        }
        if (kTurns) {
          if (grew || i == 0) refs[row] = ref;
          __syncwarp();
          pass_turn();
        }
        if (grew && i > 0) {
          wait_product(gl, 227);
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < kScale; cc += 16) {
            uint32_t o[16];
            tmem_ld16(ocol + cc, o);
            tmem_wait_ld16(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
            tmem_st16(ocol + cc, o);
            tmem_wait_st();
          }
        }
        const float r = ref == -INFINITY ? 0.f : ref;
        const float2 c22 = make_float2(c2, c2), r22 = make_float2(-r, -r);
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t p[32];
#pragma unroll
        for (int c = 0; c < kCols; c += 64) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float2 x = __ffma2_rn(make_float2(__uint_as_float(v[c + 2 * e]), __uint_as_float(v[c + 2 * e + 1])), c22, r22);
            x.x = ex2(x.x), x.y = ex2(x.y);
            acc[e & 1] = __fadd2_rn(acc[e & 1], x);
            p[e] = pack2(x.x, x.y);
          }
          if (c == 0) {
            // P's place is free once the product of S tile g - 2 has read it (P in S's place: as S was there). A parity
            // wait tells only consecutive phases apart: who waits for a tile's product has to know of the one four tiles
            // before. So every product up to g - 2 is awaited, in order; none from g on can be done before this P is there.
            if (kTurns && g >= 3) wait_product(g - 3, 229);
            if (kOwnP && g >= 2) wait_product(g - 2, 229);
            if (kOwnP) tc_fence_after();
          }
          tmem_st32(pl + half * 32 + c / 2, p);
          if (c + 64 < kCols) tmem_wait_st();  // (the store reads its registers as it goes)
        }
        acc[0] = __fadd2_rn(acc[0], acc[1]);
        sum += acc[0].x + acc[0].y;
        tmem_wait_st();
        keep(p);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(pready(g & 1u));
        if (!kOwnP && g >= 2) wait_product(g - 2, 229);
      }
      g0 += n * QT;
      // output: a row's dims, or half of them
      {
        const uint32_t gl = g0 - QT + q;
        const uint32_t ocol = tmem + lanes + 256 + q * DIM + ohalf * kOCols;
        float tot = sum;
        if (kHalves) tot += exchange(sum);
        if (kTurns) {
          const float sum2 = exchange(sum), ref2 = exchange(ref), to = fmaxf(ref, ref2);
          const float a1 = ref == to ? sum : sum * ex2(ref - to), a2 = ref2 == to ? sum2 : sum2 * ex2(ref2 - to);
          tot = wg ? a2 + a1 : a1 + a2;
          ref = to;
        }
        const float inv = tot != 0.f ? 1.f / tot : 0.f;
        const float lse = tot != 0.f ? ref + log2f(tot) : -INFINITY;
        wait_product(gl, 228);
        tc_fence_after();
        const int r = q * 128 + row;
        const bool valid = r < s.n_rows, part = s.part >= 0;
        const int rr = min(s.row0 + r, s.last), t = m.token(rr);
        const long long at = (long long)(s.first + t) * a.heads + (m.h0 + s.head) * a.group + rr - t * a.group;
        const long long prow = (long long)s.part * C::kRows + r;
#pragma unroll 1
        for (int cc = 0; cc < kOCols; cc += 32) {
          uint32_t o[32];
          tmem_ld32(ocol + cc, o);
          tmem_wait_ld32(o);
          const int d = ohalf * kOCols + cc;
          if (part) {
            float* dst = m.part_o + prow * DIM + d;
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
#pragma unroll
            for (int e = 0; e < 32; e += 8) st_v8(dst + e, o + e);
          } else if (valid) {
            uint16_t* dst = a.out + at * DIM + d;
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              o[e / 2] = pack2(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
            if (wide) {
              st_v8(dst, o), st_v8(dst + 16, o + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<uint4*>(dst + 2 * e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
        }
        if (ohalf == 0) {
          if (part)
            m.part_lse[prow] = lse;
          else if (valid && a.lse)
            a.lse[at] = lse * 0.6931471805599453f;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first(ofree);
      if (s.part >= 0 && m.join) {
        // the part is written; whoever completes the count joins all parts of this CTA's rows, in the order of the pairs
        __threadfence();
        int* last = reinterpret_cast<int*>(gbase + C::kOffMisc + 8);
        asm volatile("bar.sync 1, %0;" ::"n"(kSoftWarps * 32) : "memory");
        if (threadIdx.x == 0) {
          wait(info_bar(sg), (sg / kDescs) & 1u, 238);
          const PartInfo i = infos[sg % kDescs];
          *last = ok && atomicAdd(m.arrived + 2 * i.c0 + (s.part & 1), 1) == i.parts - 1;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kSoftWarps * 32) : "memory");
        if (*last) {
          const PartInfo info = infos[sg % kDescs];
          __threadfence();
          // A warp joins rows warp, warp + 8, ..., lane l holding the maximum and sum of row warp + 8 l, and takes the
          // rows' values in batches with all of a part's loads in flight.
          constexpr int kV = DIM / 128 + (DIM < 128), kBatch = DIM == 256 ? 4 : 8;
          const bool mine = DIM >= 128 || lane < DIM / 4;  // DIM 64: half of the lanes hold a row
          const int my_row = warp + kSoftWarps * lane;
          const bool has_row = my_row < s.n_rows;
          // parts in order: fn(row of the part buffers at which the part begins)
          auto each_part = [&](auto&& fn) {
            for (int c = info.c0, from = 0; c <= info.c1; ++c) {
              const int to = tiles_before(m.range[c + 1].begin, s.u0, s.n);
              if (to > from) fn((2 * (2ll * c + (from > 0)) + (s.part & 1)) * C::kRows);
              from = to;
            }
          };
          float top = -INFINITY, tot = 0.f;
          each_part([&](long long at) { top = has_row ? fmaxf(top, __ldcg(m.part_lse + at + my_row)) : top; });
          const float r0 = top == -INFINITY ? 0.f : top;
          each_part([&](long long at) { tot += has_row ? ex2(__ldcg(m.part_lse + at + my_row) - r0) : 0.f; });
          const float inv = tot != 0.f ? 1.f / tot : 0.f;
          const int rr = min(s.row0 + my_row, s.last), t = m.token(rr);
          const long long my_at = (long long)(s.first + t) * a.heads + (m.h0 + s.head) * a.group + rr - t * a.group;
          if (has_row && a.lse) a.lse[my_at] = tot != 0.f ? (top + log2f(tot)) * 0.6931471805599453f : -INFINITY;
          for (int b0 = 0; warp + kSoftWarps * b0 < s.n_rows; b0 += kBatch) {
            float4 o[kBatch][kV];
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
#pragma unroll
              for (int k = 0; k < kV; ++k) o[b][k] = make_float4(0.f, 0.f, 0.f, 0.f);
            each_part([&](long long at) {
              const float w = has_row ? ex2(__ldcg(m.part_lse + at + my_row) - r0) * inv : 0.f;
              float4 v[kBatch][kV];
#pragma unroll
              for (int b = 0; b < kBatch; ++b) {
                const int r = warp + kSoftWarps * (b0 + b);
#pragma unroll
                for (int k = 0; k < kV; ++k)
                  v[b][k] = mine && r < s.n_rows ? __ldcg(reinterpret_cast<const float4*>(m.part_o + (at + r) * DIM) + lane + 32 * k)
                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
              }
#pragma unroll
              for (int b = 0; b < kBatch; ++b) {
                const float wb = __shfl_sync(~0u, w, (b0 + b) & 31);
#pragma unroll
                for (int k = 0; k < kV; ++k)
                  o[b][k].x += wb * v[b][k].x, o[b][k].y += wb * v[b][k].y, o[b][k].z += wb * v[b][k].z, o[b][k].w += wb * v[b][k].w;
              }
            });
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
              const long long at = __shfl_sync(~0u, my_at, (b0 + b) & 31);
              if (mine && warp + kSoftWarps * (b0 + b) < s.n_rows)
#pragma unroll
                for (int k = 0; k < kV; ++k)
                  *reinterpret_cast<uint2*>(a.out + at * DIM + 4 * (lane + 32 * k)) =
                      make_uint2(pack2(o[b][k].x, o[b][k].y), pack2(o[b][k].z, o[b][k].w));
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  __syncwarp();
  pair_sync();  // nothing of the other CTA reads or arrives here any more
  if (warp == kWarpMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Joins the parts of divided row tiles: out = sum_p 2^(lse_p - max) o_p /
// sum_p 2^(lse_p - max). CTA (row tile, eight of its rows, kv head), a warp per
// row, several parts' loads in flight.
template <int DIM>
__global__ void __launch_bounds__(256) attention_many_combine_kernel(const ManyArgs m) {
  griddep_wait();
  constexpr int kRows = ManyCfg<DIM>::kRows, kV = DIM / 128 + (DIM < 128);
  constexpr int kBatch = DIM == 256 ? 4 : 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rt = blockIdx.x, head = blockIdx.z, pr = blockIdx.y * 8 + warp;  // row of the pair
  if (rt >= m.plan->row_tiles) return;
  const RowTile t = m.row_tile[rt];
  const int last = t.n_new * m.a.group - 1, rr = t.row0 + pr;
  if (rr > last) return;
  const long long units = m.plan->units, u0 = head * units + m.unit_off[rt], u1 = head * units + m.unit_off[rt + 1];
  // the pair that holds the first key tile: the last one whose units begin at or before it
  int lo = 0, hi = m.pairs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (m.range[mid].begin <= u0 + kTileCost)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int c0 = lo;
  if (m.range[c0 + 1].begin >= u1) return;  // one pair has all of it, and wrote the output
  int c1 = c0 + 1;
  hi = m.pairs - 1;  // the last pair with a unit before u1
  while (c1 < hi) {
    const int mid = (c1 + hi + 1) >> 1;
    if (m.range[mid].begin < u1)
      c1 = mid;
    else
      hi = mid - 1;
  }
  const int parts = c1 - c0 + 1, rank = pr / kRows, r = pr % kRows;
  // part p is pair c0 + p's: in its slot 1 if it begins inside the row tile, as all but the first do
  auto at = [&](int p) { return (2 * (2ll * (c0 + p) + (p > 0)) + rank) * kRows + r; };
  float top = -INFINITY;
  for (int p = lane; p < parts; p += 32) top = fmaxf(top, m.part_lse[at(p)]);
#pragma unroll
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, off));
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  float4 o[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool mine = DIM >= 128 || lane < DIM / 4;
  for (int p0 = 0; p0 < parts; p0 += 32) {
    const int some = min(32, parts - p0);
    const float w = lane < some ? ex2(m.part_lse[at(p0 + lane)] - ref) : 0.f;
    for (int p = 0; p < some; p += kBatch) {
      float4 v[kBatch][kV];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int k = 0; k < kV; ++k)
          v[i][k] = mine && p + i < some ? reinterpret_cast<const float4*>(m.part_o + at(p0 + p + i) * DIM)[lane + 32 * k]
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float wi = __shfl_sync(~0u, w, p + i);
        sum += wi;
#pragma unroll
        for (int k = 0; k < kV; ++k)
          o[k].x += wi * v[i][k].x, o[k].y += wi * v[i][k].y, o[k].z += wi * v[i][k].z, o[k].w += wi * v[i][k].w;
      }
    }
  }
  const int tok = m.token(rr);
  const long long dst = (long long)(t.first + tok) * m.a.heads + (m.h0 + head) * m.a.group + rr - tok * m.a.group;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  if (mine)
#pragma unroll
    for (int k = 0; k < kV; ++k)
      *reinterpret_cast<uint2*>(m.a.out + dst * DIM + 4 * (lane + 32 * k)) =
          make_uint2(pack2(o[k].x * inv, o[k].y * inv), pack2(o[k].z * inv, o[k].w * inv));
  if (lane == 0 && m.a.lse) m.a.lse[dst] = sum != 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// ---- host ---------------------------------------------------------------------------------

// Expanded tiles of one pass take at most this, if one sequence's kv head
// fits: the step runs as passes over kv heads, then over sequences.
constexpr size_t kPassBytes = size_t(2) << 30;

size_t al256(size_t v) { return (v + 255) & ~size_t(255); }

struct ManyPlan {
  int rows, tiles_max, nb, nh, pairs, max_row_tiles;  // rows: of a row tile, both CTAs'
  size_t kx, vx, bad, plan, unit_off, row_tile, range, arrived, part_o, part_lse, total;
};

// The workspace grows with every bound on the step, so that one sized for a
// larger step serves a smaller one: what depends on how the passes divide it
// has the place of the most that any division of a smaller step could use.
ManyPlan plan(const AttnArgs& a) {
  ManyPlan p{};
  const int dim = a.kv.dim;
  p.rows = dim == 64 ? 512 : 256;
  long long keys = a.kv.max_kv;
  if (a.window > 0)
    keys = std::min<long long>(keys, (long long)a.window + std::min(a.sinks, a.kv.max_kv) + a.kv.max_new + 2 * kBK);
  p.tiles_max = std::max(1, int((keys + kBK - 1) / kBK));
  const size_t head_bytes = size_t(p.tiles_max) * kBK * dim * 2 * 2;  // keys and values of a (sequence, kv head)
  const size_t fit = std::max<size_t>(1, kPassBytes / head_bytes);
  p.nh = int(std::min<size_t>(a.kv.kv_heads, fit));
  p.nb = int(std::min<size_t>(a.kv.n_seqs, std::max<size_t>(1, fit / p.nh)));
  p.pairs = num_sms() / 2;
  p.max_row_tiles = int(((long long)a.kv.n_tokens * a.group + p.rows - 1) / p.rows + p.nb);
  size_t o = 0;
  auto put = [&](size_t bytes) {
    const size_t at = o;
    o = al256(o + bytes);
    return at;
  };
  const size_t tile_bytes = head_bytes / p.tiles_max;
  const size_t pass_tiles = std::max<size_t>(p.tiles_max, kPassBytes / tile_bytes);  // at least nb nh tiles_max
  const size_t seq_tiles = size_t(a.kv.n_seqs) * p.tiles_max, tiles = std::min(seq_tiles * a.kv.kv_heads, pass_tiles);
  const size_t row_tiles = size_t(p.max_row_tiles - p.nb) + a.kv.n_seqs;
  p.kx = put(tiles * tile_bytes / 2);
  p.vx = put(tiles * tile_bytes / 2);
  p.bad = put(std::min(seq_tiles, pass_tiles));  // (with a byte per head, which moves the arrays behind: windowed prompts 1 us slower)
  p.plan = put(sizeof(PlanHdr));
  p.unit_off = put((row_tiles + 1) * 8);
  p.row_tile = put(row_tiles * sizeof(RowTile));
  p.range = put((size_t(p.pairs) + 1) * sizeof(PairRange));
  p.arrived = put(size_t(p.pairs) * 2 * 4);
  p.part_o = put(size_t(2) * p.pairs * p.rows * dim * 4);
  p.part_lse = put(size_t(2) * p.pairs * p.rows * 4);
  p.total = o;
  return p;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_beside(const KvCall& c, const char* name, void (*kernel)(KArgs...), dim3 grid, int block, size_t smem,
                          int cluster, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...)) return e;
  return c.launched(name);
}

template <int DIM>
cudaError_t launch(ManyArgs m, const ManyPlan& p, const KvCall& c) {
  using C = ManyCfg<DIM>;
  if (!ensure_smem_limit(reinterpret_cast<const void*>(&attention_many_kernel<DIM>), C::kSmem)) return cudaErrorInvalidValue;
  for (m.b0 = 0; m.b0 < m.a.kv.n_seqs; m.b0 += p.nb)
    for (m.h0 = 0; m.h0 < m.a.kv.kv_heads; m.h0 += p.nh) {
      m.nb = std::min(p.nb, m.a.kv.n_seqs - m.b0);
      m.nh = std::min(p.nh, m.a.kv.kv_heads - m.h0);
      const long long grid = 1 + 2ll * m.nb * m.nh * p.tiles_max;
      if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
      attention_expand_kernel<DIM><<<unsigned(grid), kPlanThreads, 0, c.stream>>>(m);
      if (cudaError_t e = c.launched("attention_expand")) return e;
      if (cudaError_t e = launch_beside(c, "attention_many", attention_many_kernel<DIM>, dim3(2 * p.pairs), kThreads,
                                        C::kSmem, 2, m))
        return e;
      if (!m.join)
        if (cudaError_t e = launch_beside(c, "attention_many_combine", attention_many_combine_kernel<DIM>,
                                          dim3(p.max_row_tiles, C::kPairRows / 8, m.nh), 256, 0, 1, m))
          return e;
    }
  return cudaSuccess;
}

}  // namespace

size_t attention_many_workspace(const AttnArgs& a) { return a.kv.n_seqs > 0 ? plan(a).total : 0; }

cudaError_t attention_many(const AttnArgs& a, int max_few, void* ws, const KvCall& c) {
  const ManyPlan p = plan(a);
  uint8_t* w = static_cast<uint8_t*>(ws);
  ManyArgs m{};
  m.a = a;
  m.max_few = max_few;
  m.tiles_max = p.tiles_max;
  m.kx = w + p.kx;
  m.vx = w + p.vx;
  m.bad = w + p.bad;
  m.plan = reinterpret_cast<PlanHdr*>(w + p.plan);
  m.unit_off = reinterpret_cast<long long*>(w + p.unit_off);
  m.row_tile = reinterpret_cast<RowTile*>(w + p.row_tile);
  m.range = reinterpret_cast<PairRange*>(w + p.range);
  m.max_row_tiles = p.max_row_tiles;
  m.pairs = p.pairs;
  // Parts of a row tile are about pairs / row tiles. Up to two are joined in
  // the kernel, by the CTA that writes the last; more of them by the combine
  // kernel, over all of the GPU. Combined against joined in the kernel, us, 16
  // heads over 2 of 128 dims, one sequence over 8000 keys: 8 row tiles 29 and
  // 41, 32 of them 43 and 46, 64 of them 70 and 67; the 256 row tiles of a
  // prompt of 4096 86 and 72. Of 256 dims, 8 row tiles 35 and 63.
  const long long row_tiles = std::max(1ll, (long long)a.kv.n_tokens * a.group / p.rows) * a.kv.kv_heads;
  m.join = row_tiles * 2 >= p.pairs;
  m.arrived = reinterpret_cast<int*>(w + p.arrived);
  m.part_o = reinterpret_cast<float*>(w + p.part_o);
  m.part_lse = reinterpret_cast<float*>(w + p.part_lse);
  m.inv_group = ((1ull << 32) + a.group - 1) / a.group;
  return a.kv.dim == 64 ? launch<64>(m, p, c) : a.kv.dim == 128 ? launch<128>(m, p, c) : launch<256>(m, p, c);
}

}  // namespace moe
