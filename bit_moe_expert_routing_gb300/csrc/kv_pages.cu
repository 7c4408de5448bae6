// The pages of a set of sequences, kept on the device: given, taken back,
// shared by forks, copied before a write, moved together.
//
// A plan is made by one CTA (the tables of a step are some 10 to 100 KB, and
// what counts is that no host waits for it); the pages that it moves are then
// copied by a grid of the size of the GPU, in all caches that share the set,
// which finds their number on the device.
#include "kv_host.cuh"

namespace moe {
namespace {

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kChunk = 4 * kPlanThreads;  // references scanned at a time
constexpr int kCopyThreads = 256;
constexpr int kMaxCaches = 64;  // of one copy launch (a kernel's arguments hold 4 KB)
constexpr int kPageBad = 203;   // detail of a page error in the status word

struct PagesArgs {
  int n_pages, page_bits, n_seqs, columns;
  int32_t* table;
  int32_t* held;
  int32_t* refs;
  WsHeader* hdr;
  // scratch
  int32_t* count;  // [0] moves, [1] pages from this one on have moved (compaction)
  int32_t* src;    // [n_pages] moves
  int32_t* dst;    // [n_pages]
  int32_t* list;   // [n_pages] free pages; new places (compaction)
  int32_t* want;   // [n_seqs] pages that a sequence wants
};

// The step's part of an update.
struct StepArgs {
  const int32_t* q_off;
  const int32_t* kv_len;
  int max_new, max_kv;
};

__device__ __forceinline__ bool is_page(const PagesArgs& a, int p) { return unsigned(p) < unsigned(a.n_pages); }

// Sum over the CTA of the values before this thread's; *total gets the sum of
// all. (buf: kPlanWarps ints; the CTA is together before and after.)
__device__ __forceinline__ int scan_before(int v, int* total, int* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int s = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(~0u, s, off);
    if (lane >= off) s += u;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = s;
  __syncthreads();
  static_assert(kPlanWarps == 32, "a lane per warp");
  int w = buf[lane];  // sums of the warps up to each
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(~0u, w, off);
    if (lane >= off) w += u;
  }
  *total = __shfl_sync(~0u, w, 31);
  const int before = __shfl_sync(~0u, w, max(warp, 1) - 1);
  return (warp ? before : 0) + s - v;
}

// References of pages p .. p + 3 (p a multiple of 4); past the last page: in use.
__device__ __forceinline__ int4 refs4(const PagesArgs& a, int p) {
  if (p + 4 <= a.n_pages) return __ldcg(reinterpret_cast<const int4*>(a.refs + p));
  int4 r = make_int4(1, 1, 1, 1);
  if (p < a.n_pages) r.x = __ldcg(a.refs + p);
  if (p + 1 < a.n_pages) r.y = __ldcg(a.refs + p + 1);
  if (p + 2 < a.n_pages) r.z = __ldcg(a.refs + p + 2);
  return r;
}

// What a step wants of sequence b: pages that it needs, the first one that it writes. False: it is not to be touched.
__device__ __forceinline__ bool wants(const PagesArgs& a, const StepArgs& s, int b, int* need, int* first) {
  const int kv = s.kv_len[b], n = s.q_off[b + 1] - s.q_off[b];
  const int size = 1 << a.page_bits;
  if (kv < 0 || kv > s.max_kv || n < 0 || n > s.max_new || (kv + size - 1) >> a.page_bits > a.columns) return false;
  *need = (kv + size - 1) >> a.page_bits;
  *first = n > 0 ? max(kv - n, 0) >> a.page_bits : a.columns;
  return true;
}

// One CTA. A page that is to be copied is marked in the table as -2 - page
// between the count of what is wanted and the giving.
__global__ void __launch_bounds__(kPlanThreads) pages_update_kernel(const PagesArgs a, const StepArgs s) {
  __shared__ int buf[kPlanWarps];
  __shared__ int n_free_s, n_moves;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) n_moves = 0;

  // pages go back
  for (int b = warp; b < a.n_seqs; b += kPlanWarps) {
    int need, first;
    if (!wants(a, s, b, &need, &first)) {
      if (lane == 0) report(a.hdr, MOE_ERR_DEVICE_CHECK, kPageBad);
      continue;
    }
    int32_t* row = a.table + (long long)b * a.columns;
    const int held = min(a.held[b], a.columns);
    for (int j = need + lane; j < held; j += 32) {
      const int p = row[j];
      if (is_page(a, p)) atomicAdd(a.refs + p, -1);
      row[j] = -1;
    }
    __syncwarp();  // every lane has read held
    if (lane == 0 && need < held) a.held[b] = need;
  }
  __syncthreads();
  // what every sequence wants
  for (int b = warp; b < a.n_seqs; b += kPlanWarps) {
    int need, first, n = 0;
    if (wants(a, s, b, &need, &first)) {
      int32_t* row = a.table + (long long)b * a.columns;
      const int held = max(0, min(__ldcg(a.held + b), a.columns));
      for (int j = first + lane; j < held; j += 32) {
        const int p = row[j];
        if (is_page(a, p) && __ldcg(a.refs + p) > 1) row[j] = -2 - p, ++n;
      }
      n = __reduce_add_sync(~0u, n) + max(0, need - held);
    }
    if (lane == 0) a.want[b] = n;
  }
  __syncthreads();
  // where each sequence's pages begin among those given
  int total = 0;
  for (int b0 = 0; b0 < a.n_seqs; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int sum;
    const int before = scan_before(b < a.n_seqs ? a.want[b] : 0, &sum, buf);
    if (b < a.n_seqs) a.want[b] = total + before;
    total += sum;
    __syncthreads();
  }
  // the first `total` free pages
  int n_free = 0;
  for (int p0 = 0; p0 < a.n_pages && n_free < total; p0 += kChunk) {
    const int p = p0 + 4 * threadIdx.x;
    const int4 r = refs4(a, p);
    const int n = (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    int sum;
    int at = n_free + scan_before(n, &sum, buf);
    if (r.x == 0) a.list[at++] = p;
    if (r.y == 0) a.list[at++] = p + 1;
    if (r.z == 0) a.list[at++] = p + 2;
    if (r.w == 0) a.list[at++] = p + 3;
    n_free += sum;
    __syncthreads();
  }
  if (threadIdx.x == 0) n_free_s = n_free;
  __syncthreads();
  // the giving
  for (int b = warp; b < a.n_seqs; b += kPlanWarps) {
    const int at0 = __ldcg(a.want + b), at1 = b + 1 < a.n_seqs ? __ldcg(a.want + b + 1) : total;
    if (at0 == at1) continue;  // (a sequence that is not to be touched wants nothing)
    int need, first;
    wants(a, s, b, &need, &first);
    int32_t* row = a.table + (long long)b * a.columns;
    const int held = max(0, min(__ldcg(a.held + b), a.columns));
    const bool fits = at1 <= n_free_s;
    if (!fits && lane == 0) report(a.hdr, MOE_ERR_DEVICE_CHECK, kPageBad);
    int at = at0;
    for (int j0 = min(first, held); j0 < held; j0 += 32) {
      const int j = j0 + lane, p = j < held ? -2 - __ldcg(row + j) : -1;
      const bool marked = p >= 0 && is_page(a, p);
      const unsigned m = __ballot_sync(~0u, marked);
      if (marked) {
        atomicAdd(a.refs + p, -1);
        int to = -1;
        if (fits) {
          to = __ldcg(a.list + at + __popc(m & ((1u << lane) - 1)));
          a.refs[to] = 1;
          const int i = atomicAdd(&n_moves, 1);
          a.src[i] = p;
          a.dst[i] = to;
        }
        row[j] = to;
      }
      at += __popc(m);
    }
    if (!fits) continue;
    for (int j = held + lane; j < need; j += 32) {
      const int to = __ldcg(a.list + at + j - held);
      row[j] = to;
      a.refs[to] = 1;
    }
    __syncwarp();  // every lane has read held
    if (lane == 0 && need > held) a.held[b] = need;
  }
  __syncthreads();
  if (threadIdx.x == 0) a.count[0] = n_moves, a.count[1] = a.n_pages;
}

// One CTA: which pages move where.
__global__ void __launch_bounds__(kPlanThreads) pages_compact_kernel(const PagesArgs a) {
  __shared__ int buf[kPlanWarps];
  int live = 0;
  for (int p0 = 0; p0 < a.n_pages; p0 += kChunk) {
    const int4 r = refs4(a, p0 + 4 * threadIdx.x);
    live += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
  }
  // (past the last page refs4 says 1)
  const int past = (a.n_pages + kChunk - 1) / kChunk * kChunk - a.n_pages;
  int sum;
  scan_before(live, &sum, buf);
  live = sum - past;
  __syncthreads();
  int n_src = 0, n_dst = 0;
  for (int p0 = 0; p0 < a.n_pages; p0 += kChunk) {
    const int p = p0 + 4 * threadIdx.x;
    const int4 r = refs4(a, p);
    const int v[4] = {r.x, r.y, r.z, r.w};
    int n = 0;  // sources in the high half, destinations in the low
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool is = p + i < a.n_pages && (p + i < live ? v[i] <= 0 : v[i] > 0);
      n += is ? (p + i < live ? 1 : 1 << 16) : 0;
    }
    int all;
    const int before = scan_before(n, &all, buf);
    int s = n_src + (before >> 16), d = n_dst + (before & 0xFFFF);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p + i >= a.n_pages) break;
      if (p + i < live) {
        if (v[i] <= 0) a.dst[d++] = p + i;
      } else {
        if (v[i] > 0) a.src[s++] = p + i;
        a.list[p + i] = p + i;
      }
    }
    n_src += all >> 16;
    n_dst += all & 0xFFFF;
    __syncthreads();
  }
  for (int i = threadIdx.x; i < n_src; i += kPlanThreads) {  // (as many places below as pages above)
    const int from = __ldcg(a.src + i), to = __ldcg(a.dst + i);
    a.list[from] = to;
    a.refs[to] = __ldcg(a.refs + from);
    a.refs[from] = 0;
  }
  if (threadIdx.x == 0) a.count[0] = n_src, a.count[1] = live;
}

struct CopyArgs {
  uint32_t* codes[kMaxCaches][2];
  uint16_t* scales[kMaxCaches][2];
  uint16_t* biases[kMaxCaches][2];
  int n_caches, n_pages;
  int codes16, sb16;       // 16-byte words of a page's codes; of its scales, or biases (keys' or values')
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;    // on the device; NULL: n
  int n;
  WsHeader* hdr;
  int32_t* table;          // compaction: entries past count[1] become list's; NULL: none
  const int32_t* list;
  long long entries;
};

// A thread's 16 bytes of a page of a cache, at word `x` of the page's six arrays.
__device__ __forceinline__ uint4* word_of(const CopyArgs& c, int cache, int page, int x) {
  const int half = c.codes16 + 2 * c.sb16, kv = x >= half;
  x -= kv ? half : 0;
  if (x < c.codes16) return reinterpret_cast<uint4*>(c.codes[cache][kv]) + (long long)page * c.codes16 + x;
  x -= c.codes16;
  uint16_t* p = x < c.sb16 ? c.scales[cache][kv] : c.biases[cache][kv];
  return reinterpret_cast<uint4*>(p) + (long long)page * c.sb16 + (x < c.sb16 ? x : x - c.sb16);
}

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ CopyArgs c) {
  constexpr int kWords = 4;  // of a thread, in flight together
  if (c.table) {
    const int from = c.count[1];
    for (long long i = blockIdx.x * kCopyThreads + threadIdx.x; i < c.entries; i += (long long)gridDim.x * kCopyThreads) {
      const int p = c.table[i];
      if (p >= from && p < c.n_pages) c.table[i] = c.list[p];
    }
  }
  const int n = c.count ? c.count[0] : c.n;
  const int words = 2 * (c.codes16 + 2 * c.sb16), pieces = (words + kWords * kCopyThreads - 1) / (kWords * kCopyThreads);
  const long long units = (long long)n * c.n_caches * pieces;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int piece = int(u % pieces);
    const long long v = u / pieces;
    const int cache = int(v % c.n_caches), move = int(v / c.n_caches);
    const int from = c.src[move], to = c.dst[move];
    if (unsigned(from) >= unsigned(c.n_pages) || unsigned(to) >= unsigned(c.n_pages)) {
      if (threadIdx.x == 0) report(c.hdr, MOE_ERR_DEVICE_CHECK, kPageBad);
      continue;
    }
    if (from == to) continue;
    uint4 x[kWords];
    const int x0 = piece * kWords * kCopyThreads + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      if (x0 + i * kCopyThreads < words) x[i] = *word_of(c, cache, from, x0 + i * kCopyThreads);
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      if (x0 + i * kCopyThreads < words) *word_of(c, cache, to, x0 + i * kCopyThreads) = x[i];
  }
}

// CTA per pair.
constexpr int kForkThreads = 128;
__global__ void __launch_bounds__(kForkThreads) pages_fork_kernel(const PagesArgs a, const int32_t* src, const int32_t* dst,
                                                                  int n) {
  const int i = blockIdx.x, from = src[i], to = dst[i];
  bool bad = unsigned(from) >= unsigned(a.n_seqs) || unsigned(to) >= unsigned(a.n_seqs);
  for (int j = threadIdx.x; j < n; j += kForkThreads) bad |= (j < i && dst[j] == to) || src[j] == to;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) report(a.hdr, MOE_ERR_DEVICE_CHECK, kPageBad);
    return;
  }
  // (nothing else in this launch changes either sequence: `to` is this pair's alone, `from` no pair's destination)
  if (a.held[to] != 0) {
    if (threadIdx.x == 0) report(a.hdr, MOE_ERR_DEVICE_CHECK, kPageBad);
    return;
  }
  const int held = max(0, min(a.held[from], a.columns));
  for (int j = threadIdx.x; j < held; j += kForkThreads) {
    const int p = a.table[(long long)from * a.columns + j];
    a.table[(long long)to * a.columns + j] = p;
    if (is_page(a, p)) atomicAdd(a.refs + p, 1);
  }
  __syncthreads();
  if (threadIdx.x == 0) a.held[to] = held;
}

constexpr int kMaxPages = 1 << 28, kMaxSeqs = 65535;

moe_status make_pages(const moe_kv_pages* p, PagesArgs* a) {
  if (!p) return MOE_ERR_ARG;
  if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1))) return MOE_ERR_SHAPE;
  if (p->n_pages < 1 || p->n_pages > kMaxPages || p->n_seqs < 1 || p->n_seqs > kMaxSeqs || p->columns < 1 ||
      p->columns > (1 << 20))
    return MOE_ERR_SHAPE;
  const void* arrays[] = {p->table, p->held, p->refs, p->scratch};
  for (const void* q : arrays)
    if (!q || !aligned(q, 16)) return MOE_ERR_ARG;
  if (!p->status || !aligned(p->status, 256)) return MOE_ERR_ARG;
  *a = PagesArgs{p->n_pages, __builtin_ctz(p->page_size), p->n_seqs, p->columns, p->table, p->held, p->refs,
                 static_cast<WsHeader*>(p->status)};
  a->count = p->scratch;
  a->src = a->count + 4;
  a->dst = a->src + p->n_pages;
  a->list = a->dst + p->n_pages;
  a->want = a->list + p->n_pages;
  return MOE_OK;
}

// The caches as arguments of the copy: all of one shape, and of n_pages pages of page_size (0: any).
moe_status check_caches(const moe_kv_cache* const* caches, int n, int n_pages, int page_size) {
  if (n < 1 || !caches) return MOE_ERR_ARG;
  const moe_kv_batch none{};
  for (int i = 0; i < n; ++i) {
    KvArgs a;
    if (moe_status s = make_args(caches[i], &none, &a)) return s;
    const moe_kv_cache &c = *caches[i], &first = *caches[0];
    if (c.n_pages != first.n_pages || c.page_size != first.page_size || c.kv_heads != first.kv_heads ||
        c.head_dim != first.head_dim || (page_size && (c.page_size != page_size || c.n_pages != n_pages)))
      return MOE_ERR_SHAPE;
  }
  return MOE_OK;
}

cudaError_t copy_pages(CopyArgs c, const moe_kv_cache* const* caches, int n_caches, const KvCall& call) {
  const moe_kv_cache& f = *caches[0];
  c.n_pages = f.n_pages;
  c.codes16 = f.kv_heads * f.page_size * f.head_dim / 32;
  c.sb16 = f.kv_heads * f.page_size * f.head_dim / 512;
  for (int i0 = 0; i0 < n_caches; i0 += kMaxCaches) {
    c.n_caches = std::min(kMaxCaches, n_caches - i0);
    for (int i = 0; i < c.n_caches; ++i) {
      const moe_kv_cache& k = *caches[i0 + i];
      c.codes[i][0] = k.k_codes, c.codes[i][1] = k.v_codes;
      c.scales[i][0] = k.k_scales, c.scales[i][1] = k.v_scales;
      c.biases[i][0] = k.k_biases, c.biases[i][1] = k.v_biases;
    }
    pages_copy_kernel<<<8 * num_sms(), kCopyThreads, 0, call.stream>>>(c);
    if (cudaError_t e = call.launched("pages_copy")) return e;
    c.table = nullptr;  // (renamed by the first launch)
  }
  return cudaSuccess;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_kv_pages_scratch(int n_pages, int n_seqs) {
  if (n_pages < 1 || n_pages > kMaxPages || n_seqs < 1 || n_seqs > kMaxSeqs) return 0;
  return 4 + size_t(3) * n_pages + n_seqs;
}

moe_status moe_kv_pages_update(const moe_kv_pages* pages, const moe_kv_batch* b, const moe_kv_cache* const* caches,
                               int n_caches, void* stream) {
  PagesArgs a;
  reset_launch_count();
  if (moe_status s = make_pages(pages, &a)) return s;
  if (moe_status s = check_caches(caches, n_caches, a.n_pages, pages->page_size)) return s;
  if (!b || b->n_seqs != a.n_seqs || b->block_table != a.table || b->table_stride != a.columns) return MOE_ERR_ARG;
  if (!b->q_off || !b->kv_len || !aligned(b->q_off, 4) || !aligned(b->kv_len, 4)) return MOE_ERR_ARG;
  if (b->max_new < 0 || b->max_kv < 0 || b->max_kv > (1 << 24)) return MOE_ERR_ARG;
  const KvCall c = begin_call(stream);
  pages_update_kernel<<<1, kPlanThreads, 0, c.stream>>>(a, StepArgs{b->q_off, b->kv_len, b->max_new, b->max_kv});
  if (cudaError_t e = c.launched("pages_update")) return status_of(e);
  CopyArgs y{};
  y.src = a.src, y.dst = a.dst, y.count = a.count, y.hdr = a.hdr;
  return status_of(copy_pages(y, caches, n_caches, c));
}

moe_status moe_kv_pages_fork(const moe_kv_pages* pages, const int32_t* src, const int32_t* dst, int n, void* stream) {
  PagesArgs a;
  reset_launch_count();
  if (moe_status s = make_pages(pages, &a)) return s;
  if (n < 0 || n > a.n_seqs) return MOE_ERR_ARG;
  if (n == 0) return MOE_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return MOE_ERR_ARG;
  const KvCall c = begin_call(stream);
  pages_fork_kernel<<<n, kForkThreads, 0, c.stream>>>(a, src, dst, n);
  return status_of(c.launched("pages_fork"));
}

moe_status moe_kv_pages_compact(const moe_kv_pages* pages, const moe_kv_cache* const* caches, int n_caches, void* stream) {
  PagesArgs a;
  reset_launch_count();
  if (moe_status s = make_pages(pages, &a)) return s;
  if (moe_status s = check_caches(caches, n_caches, a.n_pages, pages->page_size)) return s;
  const KvCall c = begin_call(stream);
  pages_compact_kernel<<<1, kPlanThreads, 0, c.stream>>>(a);
  if (cudaError_t e = c.launched("pages_compact")) return status_of(e);
  CopyArgs y{};
  y.src = a.src, y.dst = a.dst, y.count = a.count, y.hdr = a.hdr;
  y.table = a.table, y.list = a.list, y.entries = (long long)a.n_seqs * a.columns;
  return status_of(copy_pages(y, caches, n_caches, c));
}

moe_status moe_kv_copy_pages(const moe_kv_cache* const* caches, int n_caches, const int32_t* src, const int32_t* dst, int n,
                             void* stream) {
  reset_launch_count();
  if (n < 0) return MOE_ERR_ARG;
  if (moe_status s = check_caches(caches, n_caches, 0, 0)) return s;
  if (n == 0) return MOE_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return MOE_ERR_ARG;
  CopyArgs y{};
  y.src = src, y.dst = dst, y.n = n, y.hdr = static_cast<WsHeader*>(caches[0]->status);
  return status_of(copy_pages(y, caches, n_caches, begin_call(stream)));
}

}  // extern "C"
