// kv_pool.hip -- the pages of include/qgemv_kv.h: who holds which (grown, cut,
// shared, moved together) and their data's copies.
#include "kv_common.h"

#include <algorithm>

using namespace qgemv_kv;

namespace {

struct Pool {
  int32_t *tables, *lens, *refs, *used, *work;
  int64_t max_pages;
  int n_seq, n_pages, shift;
};

// The workspace, in words: how many pages are to be copied, and how many are in
// use, then lists.
constexpr int kHead = 4;

__device__ __forceinline__ int pages_of(int64_t len, int shift) { return (int)((len + (1ll << shift) - 1) >> shift); }

// A sequence's length, kept within its table.
__device__ __forceinline__ int length_of(const Pool &p, int s) {
  return (int)min((int64_t)max(p.lens[s], 0), p.max_pages << p.shift);
}

// Counts that other threads' atomics may have changed are read past the caches
// of the compute unit, which do not see them.
__device__ __forceinline__ int fresh(const int32_t *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One holder fewer of a page (-1: none): was it the last?
__device__ __forceinline__ bool let_go(const Pool &p, int page) {
  return (unsigned)page < (unsigned)p.n_pages && atomicSub(&p.refs[page], 1) == 1;
}

// Clears the bits of free pages, of the lanes of a wave at once: a sequence's
// pages often lie in a row, and 32 lanes' atomics on a word would wait for each
// other (4500 pages of 24 sequences let go by one workgroup: 55 us, so 13).
__device__ void mark_free(const Pool &p, int page, bool free) {
  const int lane = threadIdx.x & 63, word = page >> 5;
  uint64_t todo = __ballot(free);
  for (int k = 0; k < 4 && todo; ++k) {
    const int leader = __builtin_ctzll(todo), w = __builtin_amdgcn_readlane(word, leader);
    const bool mine = free && word == w;
    uint32_t bits = mine ? 1u << (page & 31) : 0;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) bits |= __shfl_xor(bits, d);
    if (lane == leader) atomicAnd(&p.used[w], (int)~bits);
    todo &= ~__ballot(mine);
    free = free && !mine;
  }
  if (free) atomicAnd(&p.used[word], (int)~(1u << (page & 31)));
}

// The bits of the pages in word w of `used` that are in use; those past the last page are not looked at.
__device__ __forceinline__ uint32_t word_of(const Pool &p, int w, uint32_t *valid) {
  const int left = p.n_pages - 32 * w;
  *valid = left >= 32 ? ~0u : left > 0 ? (1u << left) - 1 : 0;
  return left > 0 ? (uint32_t)fresh(&p.used[w]) & *valid : 0;
}

constexpr int kThreads = 1024, kWaves = kThreads / 64;

// The sum over the threads before, and *total over all of them.  Every thread of the workgroup calls it.
__device__ uint32_t scan_threads(uint32_t v, uint32_t *total) {
  __shared__ uint32_t wave[kWaves];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint32_t sum = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(sum, d);
    if (lane >= d) sum += o;
  }
  __syncthreads();  // (the last call's sums have been read)
  if (lane == 63) wave[w] = sum;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    const uint32_t x = wave[i];
    before += i < w ? x : 0;
    all += x;
  }
  *total = all;
  return before + sum - v;
}

// a[0 .. n) to the sums before each, in place; their sum.
__device__ int scan_array(int *a, int n) {
  constexpr int kEach = QG_MAX_SEQS / kThreads;
  const int first = threadIdx.x * kEach;
  int v[kEach], sum = 0;
  uint32_t total;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    v[i] = first + i < n ? a[first + i] : 0;
    sum += v[i];
  }
  int at = (int)scan_threads(sum, &total);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (first + i < n) a[first + i] = at;
    at += v[i];
  }
  __syncthreads();
  return (int)total;
}

// The last s with before[s] <= k: the one whose share k falls into (before[0] = 0).
__device__ __forceinline__ int owner_of(const int *before, int n, int k) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= k) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// Cutting, by as many workgroups as sequences and more: of 224 forks let go,
// 42 000 entries, one takes 85 us.  Then growing, by one: a step's few hundred
// sequences of which few need a page take it a handful of dependent passes over
// the lengths, and one over the bits of the pages in use where any is needed
// (200 000 pages: 25 KB).  Free pages are walked by all threads alike, whosever
// they become.  (256 sequences that take a page each: 5 us and 12.)
// ---------------------------------------------------------------------------

__global__ void __launch_bounds__(256) cut_kernel(Pool p, const int32_t *lens) {
  const int s = blockIdx.x, len = length_of(p, s), want = lens[s];
  if (want < 0 || want >= len) return;
  const int end = pages_of(len, p.shift);
  int32_t *mine = p.tables + s * p.max_pages;
  for (int e0 = pages_of(want, p.shift) + blockIdx.y * 256; e0 < end; e0 += gridDim.y * 256) {
    const int e = e0 + threadIdx.x, page = e < end ? mine[e] : -1;
    mark_free(p, page, let_go(p, page));
    if (e < end) mine[e] = -1;
  }
}

constexpr int kStays = -2;  // of a sequence's kept page

__global__ void __launch_bounds__(kThreads) resize_kernel(Pool p, const int32_t *lens) {
  __shared__ int pre[QG_MAX_SEQS], last[QG_MAX_SEQS], kept[QG_MAX_SEQS];
  __shared__ int copies;
  const int n = p.n_seq, tid = threadIdx.x;
  int32_t *src = p.work + kHead, *dst = src + n, *list = dst + n;
  if (tid == 0) copies = 0;

  // last pages that sequences want to grow into
  for (int s = tid; s < n; s += kThreads) {
    const int len = length_of(p, s), want = lens[s];
    int page = -1;
    if (want > len && pages_of(want, p.shift) <= p.max_pages && (len & ((1 << p.shift) - 1)))
      page = p.tables[s * p.max_pages + (len >> p.shift)];
    last[s] = (unsigned)page < (unsigned)p.n_pages ? page : -1;
  }
  __syncthreads();
  // pages each one needs
  bool copied[QG_MAX_SEQS / kThreads];
#pragma unroll
  for (int i = 0; i < QG_MAX_SEQS / kThreads; ++i) {
    const int s = tid + i * kThreads;
    copied[i] = false;
    if (s >= n) continue;
    kept[s] = -1;
    const int len = length_of(p, s), want = lens[s], page = last[s];
    const int64_t wide = pages_of(want, p.shift);
    int need = want > len && wide <= p.max_pages ? (int)wide - pages_of(len, p.shift) : 0;
    if (page >= 0) {
      const int refs = fresh(&p.refs[page]);
      if (refs > 1) {
        int growing = 0, first = n;
        for (int o = n - 1; o >= 0; --o)
          if (last[o] == page) {
            ++growing;
            first = o;
          }
        copied[i] = !(growing == refs && first == s);
        need += copied[i];
        if (!copied[i]) kept[s] = page;
      }
    }
    pre[s] = need;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < QG_MAX_SEQS / kThreads; ++i)
    if (tid + i * kThreads < n && !copied[i]) last[tid + i * kThreads] = -1;
  __syncthreads();
  const int total = scan_array(pre, n);

  // the free pages of the lowest numbers
  int free_pages = 0;
  if (total > 0) {
    const int words = (p.n_pages + 31) / 32;
    for (int w0 = 0; w0 < words && free_pages < total; w0 += kThreads) {
      uint32_t valid, free_bits = 0;
      if (w0 + tid < words) {
        free_bits = ~word_of(p, w0 + tid, &valid);
        free_bits &= valid;
      }
      uint32_t found, taken = 0;
      int at = free_pages + (int)scan_threads(__popc(free_bits), &found);
      for (; free_bits && at < total; free_bits &= free_bits - 1, ++at) {
        list[at] = 32 * (w0 + tid) + __builtin_ctz(free_bits);
        taken |= free_bits & -free_bits;
      }
      if (taken) atomicOr(&p.used[w0 + tid], (int)taken);
      free_pages += (int)found;
    }
    __syncthreads();
  }
  const auto share_of = [&](int s) { return (s + 1 < n ? pre[s + 1] : total) - pre[s]; };
  const auto finds_all = [&](int s) { return share_of(s) == 0 || pre[s] + share_of(s) <= free_pages; };
  // One that keeps a page writes into it from its own length on, where a longer
  // holder that finds no page for its copy has its positions: it stays.
  for (int s = tid; s < n && total > free_pages; s += kThreads) {
    if (kept[s] < 0) continue;
    const int len = length_of(p, s);
    for (int o = s + 1; o < n; ++o)
      if (last[o] == kept[s] && length_of(p, o) > len && !finds_all(o)) {
        kept[s] = kStays;
        break;
      }
  }
  __syncthreads();
  const auto grows = [&](int s) { return kept[s] != kStays && finds_all(s); };
  const int given = min(total, free_pages);
  for (int k = tid; k < given; k += kThreads) {
    const int s = owner_of(pre, n, k);
    const int page = list[k], r = k - pre[s], copied_page = last[s];
    if (!grows(s)) {  // (given to one that does not find all of its own, or stays)
      atomicAnd(&p.used[page >> 5], (int)~(1u << (page & 31)));
      continue;
    }
    const int at = pages_of(length_of(p, s), p.shift) - (copied_page >= 0) + r;
    p.tables[s * p.max_pages + at] = page;
    p.refs[page] = 1;
    if (copied_page >= 0 && r == 0) {
      atomicSub(&p.refs[copied_page], 1);  // (never the last: another holds it)
      const int i = atomicAdd(&copies, 1);
      src[i] = copied_page;
      dst[i] = page;
    }
  }
  __syncthreads();
  for (int s = tid; s < n; s += kThreads) {
    const int len = length_of(p, s), want = lens[s] < 0 ? len : lens[s];
    p.lens[s] = pages_of(want, p.shift) <= p.max_pages && grows(s) ? want : len;
  }
  if (tid == 0) p.work[0] = copies;
}

// ---------------------------------------------------------------------------
// Forks: every sequence that changes takes its source's entries to the side and
// counts itself as their holder, then all let go what they had and take the
// new entries.  A page is never counted down before it is counted up, so none
// that stays in use is freed in between.
// ---------------------------------------------------------------------------

__device__ __forceinline__ bool forks(const Pool &p, const int32_t *from, int s) {
  const int f = from[s];
  return f != s && f >= -1 && f < p.n_seq;
}

__global__ void __launch_bounds__(256) fork_take_kernel(Pool p, const int32_t *from) {
  const int s = blockIdx.x;
  if (!forks(p, from, s)) return;
  const int f = from[s], len = f < 0 ? 0 : length_of(p, f), n = pages_of(len, p.shift);
  int32_t *rows = p.work + kHead + s * p.max_pages;
  for (int e = blockIdx.y * 256 + threadIdx.x; e < n; e += gridDim.y * 256) {
    const int page = p.tables[f * p.max_pages + e];
    rows[e] = page;
    if ((unsigned)page < (unsigned)p.n_pages) atomicAdd(&p.refs[page], 1);
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) p.work[kHead + p.n_seq * p.max_pages + s] = len;
}

__global__ void __launch_bounds__(256) fork_give_kernel(Pool p, const int32_t *from) {
  const int s = blockIdx.x;
  if (!forks(p, from, s)) return;
  const int32_t *rows = p.work + kHead + s * p.max_pages;
  const int len = p.work[kHead + p.n_seq * p.max_pages + s], n = pages_of(len, p.shift);
  // the old entries end where they do: -1 behind the length
  int32_t *mine = p.tables + s * p.max_pages;
  for (int64_t e0 = blockIdx.y * 256; e0 < p.max_pages; e0 += gridDim.y * 256) {
    const int64_t e = e0 + threadIdx.x;
    const int old = e < p.max_pages ? mine[e] : -1, now = e < n ? rows[e] : -1;
    mark_free(p, old, let_go(p, old));
    if (old != now) mine[e] = now;
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) p.lens[s] = len;
}

// ---------------------------------------------------------------------------
// Pages moved together: one workgroup lists the pages in use above their number
// and the free ones below it, others copy them and rewrite tables and counts.
// ---------------------------------------------------------------------------

__device__ __forceinline__ int32_t *moves_dst(const Pool &p) { return p.work + kHead + p.n_pages / 2; }
__device__ __forceinline__ int32_t *moves_map(const Pool &p) { return p.work + kHead + 2 * (p.n_pages / 2); }

__global__ void __launch_bounds__(kThreads) moves_kernel(Pool p) {
  const int words = (p.n_pages + 31) / 32, tid = threadIdx.x;
  uint32_t count = 0, in_use, valid;
  for (int w = tid; w < words; w += kThreads) count += __popc(word_of(p, w, &valid));
  scan_threads(count, &in_use);
  const int all = (int)in_use;
  int32_t *src = p.work + kHead, *dst = moves_dst(p), *map = moves_map(p);
  int n_src = 0, n_dst = 0;
  for (int w0 = 0; w0 < words; w0 += kThreads) {
    const int w = w0 + tid;
    uint32_t from = 0, to = 0;
    if (w < words) {
      const uint32_t used = word_of(p, w, &valid);
      const int below = all - 32 * w;  // pages of this word that stay
      const uint32_t low = below >= 32 ? ~0u : below > 0 ? (1u << below) - 1 : 0;
      from = used & ~low;
      to = ~used & valid & low;
    }
    uint32_t found;  // both counts of 1024 words fit 16 bits
    const uint32_t at = scan_threads((uint32_t)__popc(from) << 16 | __popc(to), &found);
    int i = n_src + (int)(at >> 16), j = n_dst + (int)(at & 0xffff);
    for (; from; from &= from - 1) src[i++] = 32 * w + __builtin_ctz(from);
    for (; to; to &= to - 1) dst[j++] = 32 * w + __builtin_ctz(to);
    n_src += (int)(found >> 16);
    n_dst += (int)(found & 0xffff);
  }
  __syncthreads();
  for (int i = tid; i < n_src; i += kThreads) map[src[i]] = dst[i];
  if (tid == 0) {
    p.work[0] = n_src;
    p.work[1] = all;
  }
}

__global__ void __launch_bounds__(256) moved_tables_kernel(Pool p) {
  const int all = p.work[1], s = blockIdx.x;
  if (p.work[0] == 0) return;
  const int32_t *map = moves_map(p);
  const int n = pages_of(length_of(p, s), p.shift);
  int32_t *mine = p.tables + s * p.max_pages;
  for (int e = blockIdx.y * 256 + threadIdx.x; e < n; e += gridDim.y * 256) {
    const int page = mine[e];
    if (page >= all && page < p.n_pages) mine[e] = map[page];
  }
}

__global__ void __launch_bounds__(256) moved_counts_kernel(Pool p) {
  const int n = p.work[0], all = p.work[1];
  if (n == 0) return;
  const int32_t *src = p.work + kHead, *dst = moves_dst(p);
  const int first = blockIdx.x * 256 + threadIdx.x, step = gridDim.x * 256;
  for (int i = first; i < n; i += step) {
    p.refs[dst[i]] = p.refs[src[i]];
    p.refs[src[i]] = 0;
  }
  for (int w = first; w < (p.n_pages + 31) / 32; w += step) {
    const int below = all - 32 * w;
    const uint32_t low = below >= 32 ? ~0u : below > 0 ? (1u << below) - 1 : 0;
    const int left = p.n_pages - 32 * w;
    const uint32_t valid = left >= 32 ? ~0u : (1u << left) - 1;
    p.used[w] = (int)((p.used[w] & ~valid) | low);
  }
}

// ---------------------------------------------------------------------------
// Copies of pages, all layers, keys and values.  Bound by memory: 1.1 GB of pages
// of 8 layers 447 us, 5.0 TB/s read and written.  A job is up to 16 KB of one
// page's part in one layer; a part that is smaller is taken by as many lanes as it
// has 16-byte pieces.
// ---------------------------------------------------------------------------

constexpr int kPiece = 1024;  // 16-byte pieces of a job

struct Copy {
  uint8_t *k, *v;
  const int32_t *src, *dst;
  const int32_t *count;  // device, or NULL: n
  int64_t n, layer_bytes, page_bytes;
  int64_t outer_bytes, inner_bytes;  // strides of the page's axes
  int run, inner;                    // pieces of a contiguous run, runs of the inner axis
  int vecs, jobs, layers, lanes, n_pages;
};

__global__ void __launch_bounds__(256) copy_kernel(Copy c) {
  const int64_t n = c.count ? *c.count : c.n;
  const int per = 256 / c.lanes, lane = threadIdx.x & (c.lanes - 1);
  const int64_t all = n * c.layers * 2 * c.jobs;
  for (int64_t j = (int64_t)blockIdx.x * per + threadIdx.x / c.lanes; j < all; j += (int64_t)gridDim.x * per) {
    const int64_t part = j / c.jobs, pl = part >> 1;
    const int piece = (int)(j - part * c.jobs);
    const int64_t pair = pl / c.layers;
    const int layer = (int)(pl - pair * c.layers);
    const int from = c.src[pair], to = c.dst[pair];
    if ((unsigned)from >= (unsigned)c.n_pages || (unsigned)to >= (unsigned)c.n_pages) continue;
    uint8_t *base = (part & 1 ? c.v : c.k) + layer * c.layer_bytes;
    const uint8_t *s = base + from * c.page_bytes;
    uint8_t *d = base + to * c.page_bytes;
    const int end = min(c.vecs, (piece + 1) * kPiece);
    for (int v0 = piece * kPiece + lane; v0 < end; v0 += 4 * c.lanes) {
      u32x4 x[4];
      int64_t at[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = v0 + i * c.lanes;
        at[i] = -1;
        if (v >= end) continue;
        if (c.run == c.vecs) {
          at[i] = (int64_t)v * 16;
        } else {
          const int r = v / c.run, o = r / c.inner;
          at[i] = o * c.outer_bytes + (r - o * c.inner) * c.inner_bytes + (int64_t)(v - r * c.run) * 16;
        }
        x[i] = *(const u32x4 *)(s + at[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at[i] >= 0) *(u32x4 *)(d + at[i]) = x[i];
    }
  }
}

Copy copy_of(const qg_kv_cache *cache) {
  Copy c = {};
  c.k = (uint8_t *)cache->k;
  c.v = (uint8_t *)cache->v;
  c.layer_bytes = cache->layer_stride * 2;
  c.page_bytes = cache->page_stride * 2;
  c.layers = cache->n_layer;
  c.n_pages = (int)cache->n_pages;
  struct Axis {
    int64_t stride, n;
  } inner = {cache->slot_stride, cache->page_size}, outer = {cache->head_stride, cache->n_head};
  if (inner.n == 1 || (outer.n > 1 && outer.stride < inner.stride)) std::swap(inner, outer);
  int64_t run = cache->head_dim;
  if (inner.n == 1 || inner.stride == run) {
    run *= inner.n;
    inner = outer;
    outer = {0, 1};
    if (inner.n == 1 || inner.stride == run) {
      run *= inner.n;
      inner = {0, 1};
    }
  }
  c.run = (int)(run / 8);
  c.inner = (int)inner.n;
  c.inner_bytes = inner.stride * 2;
  c.outer_bytes = outer.stride * 2;
  c.vecs = (int)(c.run * inner.n * outer.n);
  c.jobs = (c.vecs + kPiece - 1) / kPiece;
  c.lanes = 1;
  while (c.lanes < 256 && c.lanes < c.vecs) c.lanes *= 2;
  return c;
}

// Copies the pairs of a pool's workspace, or n given ones.
void launch_copy(const Copy &c, hipStream_t stream) {
  constexpr int64_t kGroups = 2048;
  const int per = 256 / c.lanes;
  const int64_t all = c.n * c.layers * 2 * c.jobs;
  const int64_t groups = std::max<int64_t>(1, std::min<int64_t>(kGroups, (all + per - 1) / per));
  hipLaunchKernelGGL(copy_kernel, dim3((unsigned)groups), dim3(256), 0, stream, c);
}

int64_t pool_words(int64_t n_seq, int64_t max_pages, int64_t n_pages) {
  return kHead + std::max(n_seq * max_pages + n_seq, 2 * n_seq + 2 * n_pages);
}

int check_sizes(int64_t n_seq, int64_t max_pages, int64_t n_pages) {
  if (n_seq < 1 || n_seq > QG_MAX_SEQS || max_pages < 1 || n_pages < 1 || n_pages > QG_MAX_POOL_PAGES ||
      max_pages > 0x7fffffff / n_seq)
    return QG_E_SHAPE;
  return QG_OK;
}

int check_pool(const qg_kv_pool *p) {
  if (!p) return QG_E_NULL;
  int rc = check_sizes(p->n_seq, p->max_pages, p->n_pages);
  if (rc) return rc;
  if (p->page_size < 1 || p->page_size > 65536 || (p->page_size & (p->page_size - 1)) ||
      p->max_pages * p->page_size > kMaxCount)
    return QG_E_SHAPE;
  if (!p->tables || !p->lens || !p->refs || !p->used || !p->work) return QG_E_NULL;
  if ((uintptr_t)p->work & 15) return QG_E_ARG;
  if (p->work_bytes < qgemv_kv_pool_bytes(p->n_seq, p->max_pages, p->n_pages)) return QG_E_SIZE;
  return QG_OK;
}

int check_pool_cache(const qg_kv_pool *p, const qg_kv_cache *c) {
  int rc;
  if ((rc = check_pool(p)) || (rc = check_cache(c))) return rc;
  return c->page_size != p->page_size || c->n_pages != p->n_pages ? QG_E_SHAPE : QG_OK;
}

Pool pool_of(const qg_kv_pool *p) {
  return {p->tables, p->lens, p->refs, p->used, (int32_t *)p->work, p->max_pages, p->n_seq, (int)p->n_pages,
          log2_of(p->page_size)};
}

// Workgroups that share a table's row.
dim3 rows_grid(const qg_kv_pool *p) {
  const int64_t y = std::min<int64_t>((p->max_pages + 255) / 256, std::max<int64_t>(1, 2048 / p->n_seq));
  return dim3((unsigned)p->n_seq, (unsigned)y);
}

}  // namespace

extern "C" {

int64_t qgemv_kv_pool_bytes(int64_t n_seq, int64_t max_pages, int64_t n_pages) {
  const int rc = check_sizes(n_seq, max_pages, n_pages);
  return rc ? rc : (pool_words(n_seq, max_pages, n_pages) * 4 + 15) / 16 * 16;
}

int qgemv_kv_resize(const qg_kv_pool *pool, const qg_kv_cache *cache, const int32_t *lens, qg_stream_t stream) {
  int rc;
  if ((rc = check_pool_cache(pool, cache))) return rc;
  if (!lens) return QG_E_NULL;
  const Pool p = pool_of(pool);
  hipLaunchKernelGGL(cut_kernel, rows_grid(pool), dim3(256), 0, stream, p, lens);
  hipLaunchKernelGGL(resize_kernel, dim3(1), dim3(kThreads), 0, stream, p, lens);
  Copy c = copy_of(cache);
  c.src = p.work + kHead;
  c.dst = c.src + p.n_seq;
  c.count = p.work;
  c.n = p.n_seq;
  launch_copy(c, stream);
  KV_HIP(hipGetLastError());
  return QG_OK;
}

int qgemv_kv_fork(const qg_kv_pool *pool, const int32_t *from, qg_stream_t stream) {
  int rc;
  if ((rc = check_pool(pool))) return rc;
  if (!from) return QG_E_NULL;
  const Pool p = pool_of(pool);
  hipLaunchKernelGGL(fork_take_kernel, rows_grid(pool), dim3(256), 0, stream, p, from);
  hipLaunchKernelGGL(fork_give_kernel, rows_grid(pool), dim3(256), 0, stream, p, from);
  KV_HIP(hipGetLastError());
  return QG_OK;
}

int qgemv_kv_compact(const qg_kv_pool *pool, const qg_kv_cache *cache, qg_stream_t stream) {
  int rc;
  if ((rc = check_pool_cache(pool, cache))) return rc;
  const Pool p = pool_of(pool);
  hipLaunchKernelGGL(moves_kernel, dim3(1), dim3(kThreads), 0, stream, p);
  Copy c = copy_of(cache);
  c.src = p.work + kHead;
  c.dst = p.work + kHead + p.n_pages / 2;
  c.count = p.work;
  c.n = p.n_pages / 2;
  if (c.n > 0) {
    launch_copy(c, stream);
    hipLaunchKernelGGL(moved_tables_kernel, rows_grid(pool), dim3(256), 0, stream, p);
    const int groups = std::max(1, std::min(256, (p.n_pages + 2047) / 2048));
    hipLaunchKernelGGL(moved_counts_kernel, dim3(groups), dim3(256), 0, stream, p);
  }
  KV_HIP(hipGetLastError());
  return QG_OK;
}

int qgemv_kv_copy(const qg_kv_cache *cache, const int32_t *src, const int32_t *dst, int64_t n, qg_stream_t stream) {
  int rc;
  if ((rc = check_cache(cache))) return rc;
  if (n < 0 || n > kMaxCount) return QG_E_ARG;
  if (n == 0) return QG_OK;
  if (!src || !dst) return QG_E_NULL;
  Copy c = copy_of(cache);
  c.src = src;
  c.dst = dst;
  c.n = n;
  launch_copy(c, stream);
  KV_HIP(hipGetLastError());
  return QG_OK;
}

}  // extern "C"
