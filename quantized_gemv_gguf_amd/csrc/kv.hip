// kv.hip -- the C ABI of include/qgemv_kv.h but for attention (kv_attend.hip)
// and the pages (kv_pool.hip): argument checks, rotary positions, new tokens
// into the cache.
#include "kv_common.h"

#include <algorithm>
#include <cmath>

using namespace qgemv_kv;

namespace {

// ---------------------------------------------------------------------------
// Rotary positions.  A pair (a, b) at position p with frequency f becomes
//     (a cos t - b sin t, b cos t + a sin t) mscale,   t = p f,
// and the gradient's turn is that by -t.  Bound by memory: every value is read
// and written once (8191 tokens, 64 heads of 128, bf16: 51 us, 5.2 TB/s; a large
// copy does 5.0).  A workgroup computes the sines of its few tokens once,
// into LDS, and then walks over all their heads.  t is reduced in 64 bits to a
// quarter turn (p f passes 10^6 radians in a long context, where fp32 has
// lost the angle), sine and cosine of the rest are fp32.
// ---------------------------------------------------------------------------

constexpr int kAngles = 512;  // sines and cosines in LDS
constexpr int kToks = 16;     // most tokens of a workgroup

struct Turn {
  const double *freqs;
  double mscale;
  int half;  // pairs; 0: nothing is turned
  int interleaved;
  int inverse;
};

__device__ __forceinline__ float2 sine_of(const Turn &r, int i, int pos) {
  const double quarters = (double)pos * (r.freqs[i] * 0.63661977236758134308);  // 2 / pi
  const double whole = rint(quarters);
  const float x = (float)(quarters - whole) * 0.5f;  // in half turns: [-1/4, 1/4]
  const int n = (int)(long long)whole & 3;
  float s = sinpif(x), c = cospif(x);
  if (n & 1) {
    const float t = s;
    s = c;
    c = -t;
  }
  if (n & 2) {
    s = -s;
    c = -c;
  }
  const float m = (float)r.mscale;
  return make_float2(c * m, (r.inverse ? -s : s) * m);
}

// Unit u of a head: V pairs to turn, or where those end up to 2 V values to copy.
template <int X, int V>
__device__ __forceinline__ void head_unit(const uint8_t *src, uint8_t *dst, int type, const float2 *angles, int half,
                                          int interleaved, int dim, int u) {
  constexpr int ES = sizeof(typename Elem<X>::Raw);
  if (u * V < half) {
    float a[V], b[V];
    float2 t[V];
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = angles[u * V + i];
    if (interleaved) {
      float x[2 * V];
      load_n<X>(src + 2 * u * V * ES, x);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        a[i] = x[2 * i];
        b[i] = x[2 * i + 1];
        x[2 * i] = a[i] * t[i].x - b[i] * t[i].y;
        x[2 * i + 1] = b[i] * t[i].x + a[i] * t[i].y;
      }
      store_as(type, dst, 2 * u * V, x);
    } else {
      load_n<X>(src + u * V * ES, a);
      load_n<X>(src + (half + u * V) * ES, b);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float x = a[i] * t[i].x - b[i] * t[i].y;
        b[i] = b[i] * t[i].x + a[i] * t[i].y;
        a[i] = x;
      }
      store_as(type, dst, u * V, a);
      store_as(type, dst, half + u * V, b);
    }
    return;
  }
  const int at = 2 * half + 2 * (u - half / V) * V;
  if (at + 2 * V <= dim) {
    float x[2 * V];
    load_n<X>(src + at * ES, x);
    store_as(type, dst, at, x);
  } else {
    for (int i = at; i < dim; ++i) {
      float x[1];
      load_n<X>(src + i * ES, x);
      store_as(type, dst, i, x);
    }
  }
}

// Walks (token, head, unit) with a workgroup's threads without dividing.
struct Walk {
  int u, h, t, du, dh, dt, units, heads;
  __device__ Walk(int tid, int step, int units_, int heads_) : units(units_), heads(heads_) {
    const int q = tid / units, sq = step / units;
    u = tid - q * units;
    t = q / heads;
    h = q - t * heads;
    du = step - sq * units;
    dt = sq / heads;
    dh = sq - dt * heads;
  }
  __device__ void next() {
    u += du;
    h += dh;
    t += dt;
    if (u >= units) {
      u -= units;
      ++h;
    }
    if (h >= heads) {
      h -= heads;
      ++t;
    }
  }
};

struct RopeArgs {
  Heads x, y;
  Turn turn;
  const int32_t *pos;
  int n_tok, n_head, dim, units, toks, heads;  // heads: of one workgroup; toks: tokens of one
};

template <int X, int V> __global__ void __launch_bounds__(256) rope_kernel(RopeArgs a, int64_t group0) {
  __shared__ float2 angles[kAngles];
  const int half = a.turn.half;
  const int t0 = (int)((group0 + blockIdx.x) * a.toks), toks = min(a.toks, a.n_tok - t0);
  const int h0 = blockIdx.y * a.heads, heads = min(a.heads, a.n_head - h0);
  for (int i = threadIdx.x; i < toks * half; i += 256) angles[i] = sine_of(a.turn, i % half, a.pos[t0 + i / half]);
  __syncthreads();
  constexpr int ES = sizeof(typename Elem<X>::Raw);
  for (Walk w(threadIdx.x, 256, a.units, heads); w.t < toks; w.next()) {
    const int64_t t = t0 + w.t, h = h0 + w.h;
    head_unit<X, V>(a.x.p + (t * a.x.tok_stride + h * a.x.head_stride) * ES,
                    a.y.p + (t * a.y.tok_stride + h * a.y.head_stride) * elem_size(a.y.type), a.y.type,
                    angles + w.t * half, half, a.turn.interleaved, a.dim, w.u);
  }
}

// ---------------------------------------------------------------------------
// New tokens into the cache.  As above, over the heads of q (turned into
// q_out), k (turned into its slot) and v (copied to its slot); a workgroup
// first finds its tokens' sequences and slots.  (7 ragged prompts up to 2048
// tokens, 7948 in all, 64 heads over 8 of 128, bf16: 64 us, 5.1 TB/s.)
// ---------------------------------------------------------------------------

struct AppendArgs {
  Heads q, q_out, k, v;
  Turn turn;
  Seqs seqs;
  const int32_t *pos;
  uint8_t *ck, *cv;
  int64_t page_stride, head_stride, slot_stride;
  int64_t n_pages;
  int cache_type, n_tok, q_heads, kv_heads, dim, units, toks, heads;
};

// The last sequence that starts at row t or before, by the 64 lanes of a wave:
// -1 where the first starts behind it.
__device__ __forceinline__ int seq_of(const Seqs &q, int t) {
  int lo = -1, hi = q.n_seq;  // starts[lo] <= t < starts[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64;
    const int at = lo + step * (int)((threadIdx.x & 63) + 1);
    const uint64_t below = __ballot(at < hi && q.starts[min(at, q.n_seq)] <= t);
    // (of rising starts the lanes below come first)
    const int n = below == ~0ull ? 64 : __builtin_ctzll(~below);
    hi = min(hi, lo + step * (n + 1));
    lo += step * n;
  }
  return lo;
}

template <int X, int V> __global__ void __launch_bounds__(256) append_kernel(AppendArgs a, int64_t group0) {
  __shared__ float2 angles[kAngles];
  __shared__ int64_t slot[kToks];  // its first element in the layer, -1: nowhere
  __shared__ int at[kToks];        // the turn's position
  __shared__ bool any[kToks];
  const int half = a.turn.half;
  const int t0 = (int)((group0 + blockIdx.x) * a.toks), toks = min(a.toks, a.n_tok - t0);
  const int h0 = blockIdx.y * a.heads, heads = min(a.heads, a.q_heads + 2 * a.kv_heads - h0);
  for (int i = threadIdx.x >> 6; i < toks; i += 4) {
    const int t = t0 + i, s = seq_of(a.seqs, t);
    int64_t to = -1;
    int64_t p = 0;
    bool in = false;
    if (s >= 0) {
      int start, n, len;
      seq_rows(a.seqs, s, a.n_tok, start, n, len);
      in = t - start < n;
      p = (int64_t)len - n + (t - start);
      if (in && p >= 0 && p < room_of(a.seqs)) {
        const int64_t page = a.seqs.tables[s * a.seqs.max_pages + (p >> a.seqs.page_shift)];
        if (page >= 0 && page < a.n_pages)
          to = page * a.page_stride + (p & ((1 << a.seqs.page_shift) - 1)) * a.slot_stride;
      }
    }
    if ((threadIdx.x & 63) == 0) {
      slot[i] = to;
      at[i] = a.pos ? a.pos[t] : (int)p;
      any[i] = in;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < toks * half; i += 256) angles[i] = sine_of(a.turn, i % half, at[i / half]);
  __syncthreads();
  constexpr int ES = sizeof(typename Elem<X>::Raw);
  for (Walk w(threadIdx.x, 256, a.units, heads); w.t < toks; w.next()) {
    const int64_t t = t0 + w.t;
    const int h = h0 + w.h;
    const float2 *ang = angles + w.t * half;
    const int64_t to = slot[w.t];
    if (h < a.q_heads) {
      if (any[w.t])
        head_unit<X, V>(a.q.p + (t * a.q.tok_stride + h * a.q.head_stride) * ES,
                        a.q_out.p + (t * a.q_out.tok_stride + h * a.q_out.head_stride) * elem_size(a.q_out.type),
                        a.q_out.type, ang, half, a.turn.interleaved, a.dim, w.u);
    } else if (to >= 0) {
      const bool key = h < a.q_heads + a.kv_heads;
      const int kh = h - a.q_heads - (key ? 0 : a.kv_heads);
      const Heads &src = key ? a.k : a.v;
      if (!key && 2 * w.u * V >= a.dim) continue;  // (a turned head's units may be more than a copied one's)
      head_unit<X, V>(src.p + (t * src.tok_stride + kh * src.head_stride) * ES,
                      (key ? a.ck : a.cv) + (to + kh * a.head_stride) * 2, a.cache_type, ang, key ? half : 0,
                      a.turn.interleaved, a.dim, w.u);
    }
  }
}

// The most pairs of a unit that divide a head's into whole units, 16 bytes a
// load at least where they do.
int pairs_of(int half) { return half % 8 == 0 ? 8 : half % 4 == 0 ? 4 : 1; }

// How many tokens, or heads of one token, a workgroup takes.
void share(int64_t n_tok, int n_head, int units, int half, int &toks, int &heads, dim3 &grid) {
  // sixteen workgroups a compute unit (8191 tokens of 64 heads of 128: 51 us, with four 62;
  // with a token each 55, and 32000 tokens of one head of 64 24 instead of 7.5)
  constexpr int64_t kGroups = 4096;
  int64_t t = std::max<int64_t>(1, n_tok / kGroups);
  t = std::min<int64_t>(t, kToks);
  if (half > 0) t = std::max<int64_t>(1, std::min<int64_t>(t, kAngles / half));
  toks = (int)t;
  const int64_t groups = (n_tok + t - 1) / t;
  const int64_t parts =
      std::max<int64_t>(1, std::min<int64_t>(kGroups / groups, ((int64_t)n_head * units + 255) / 256));
  heads = (int)((n_head + parts - 1) / parts);
  grid = dim3((unsigned)groups, (unsigned)((n_head + heads - 1) / heads));
}

template <typename F> void in_grids(dim3 grid, F f) {
  for (int64_t first = 0; first < (int64_t)grid.x; first += kMaxGrid)
    f(first, dim3((unsigned)std::min<int64_t>(grid.x - first, kMaxGrid), grid.y));
}

int check_rope(const qg_rope *r, int64_t head_dim) {
  if (!r) return QG_E_NULL;
  if (r->n_rot < 2 || r->n_rot % 2 != 0 || r->n_rot > head_dim || r->n_rot > 2 * kAngles) return QG_E_SHAPE;
  if ((r->interleaved != 0 && r->interleaved != 1) || !std::isfinite(r->mscale)) return QG_E_ARG;
  if (!r->freqs) return QG_E_NULL;
  if ((uintptr_t)r->freqs & 7) return QG_E_ARG;
  return QG_OK;
}

Turn turn_of(const qg_rope *r, int inverse) {
  if (!r) return {nullptr, 1.0, 0, 0, 0};
  return {r->freqs, r->mscale, r->n_rot / 2, r->interleaved, inverse};
}

// f(kernel<X, V>) for a checked type and number of pairs.
#define QG_KV_PICK(kernel, type, pairs, f)            \
  do {                                                \
    if (type == QG_F32) {                             \
      if (pairs == 8) f((kernel<QG_F32, 8>));         \
      else if (pairs == 4) f((kernel<QG_F32, 4>));    \
      else f((kernel<QG_F32, 1>));                    \
    } else if (type == QG_F16) {                      \
      if (pairs == 8) f((kernel<QG_F16, 8>));         \
      else if (pairs == 4) f((kernel<QG_F16, 4>));    \
      else f((kernel<QG_F16, 1>));                    \
    } else {                                          \
      if (pairs == 8) f((kernel<QG_BF16, 8>));        \
      else if (pairs == 4) f((kernel<QG_BF16, 4>));   \
      else f((kernel<QG_BF16, 1>));                   \
    }                                                 \
  } while (0)

}  // namespace

// ---------------------------------------------------------------------------
// Checks
// ---------------------------------------------------------------------------

namespace qgemv_kv {

constexpr int64_t kMaxSpan = 1ll << 48;  // elements an array may span

int check_heads(const qg_heads *h, bool out, int64_t most_dim) {
  if (!h) return QG_E_NULL;
  const int es = elem_size(h->type);
  if (!es) return QG_E_FMT;
  if (h->n_tok < 0 || h->n_tok > kMaxCount || h->n_head < 1 || h->n_head > QG_MAX_HEADS || h->head_dim < 1 ||
      h->head_dim > most_dim)
    return QG_E_SHAPE;
  if (h->reserved != 0 || h->tok_stride < 0 || h->head_stride < 0 || h->tok_stride > kMaxSpan ||
      h->head_stride > kMaxSpan || (__int128)h->n_tok * h->tok_stride + (__int128)h->n_head * h->head_stride > kMaxSpan)
    return QG_E_ARG;
  if (out && h->n_tok > 0) {
    // heads within tokens, or tokens within heads
    const int64_t row = (h->n_head - 1) * h->head_stride + h->head_dim;
    const int64_t col = (h->n_tok - 1) * h->tok_stride + h->head_dim;
    const bool rows = (h->n_head == 1 || h->head_stride >= h->head_dim) && (h->n_tok == 1 || h->tok_stride >= row);
    const bool cols = (h->n_tok == 1 || h->tok_stride >= h->head_dim) && (h->n_head == 1 || h->head_stride >= col);
    if (!rows && !cols) return QG_E_ARG;
  }
  if (h->n_tok > 0 && !h->data) return QG_E_NULL;
  if ((uintptr_t)h->data & (es - 1)) return QG_E_ARG;
  return QG_OK;
}

int check_cache(const qg_kv_cache *c) {
  if (!c) return QG_E_NULL;
  if (c->type != QG_F16 && c->type != QG_BF16) return QG_E_FMT;
  if (c->page_size < 1 || c->page_size > 65536 || (c->page_size & (c->page_size - 1)) || c->n_layer < 1 ||
      c->n_layer > 65536 || c->n_head < 1 || c->n_head > QG_MAX_HEADS || c->head_dim < 32 || c->head_dim % 32 != 0 ||
      c->head_dim > QG_MAX_HEAD_DIM || c->n_pages < 1 || c->n_pages > kMaxCount)
    return QG_E_SHAPE;
  if ((int64_t)c->n_head * c->page_size * c->head_dim > 1ll << 33) return QG_E_SHAPE;  // copies count its pieces in 32 bits
  if (c->reserved != 0) return QG_E_ARG;
  // from the innermost axis out, each must step past all that is within it
  struct Axis {
    int64_t stride, n;
  } axes[4] = {{c->slot_stride, c->page_size}, {c->head_stride, c->n_head}, {c->page_stride, c->n_pages},
               {c->layer_stride, c->n_layer}};
  for (const Axis &x : axes)
    if (x.stride <= 0 || x.stride % 8 != 0 || x.stride > kMaxSpan) return QG_E_ARG;
  std::sort(axes, axes + 4, [](const Axis &x, const Axis &y) { return x.stride < y.stride; });
  __int128 extent = c->head_dim;
  for (const Axis &x : axes)
    if (x.n > 1) {
      if (x.stride < extent) return QG_E_ARG;
      extent += (__int128)(x.n - 1) * x.stride;
    }
  if (extent > kMaxSpan) return QG_E_ARG;
  if (!c->k || !c->v) return QG_E_NULL;
  if (((uintptr_t)c->k | (uintptr_t)c->v) & 15) return QG_E_ARG;
  return QG_OK;
}

int check_seqs(const qg_kv_seqs *q, const qg_kv_cache *c) {
  if (!q) return QG_E_NULL;
  if (q->n_seq < 0 || q->n_seq > QG_MAX_SEQS || q->max_pages < 0 || q->max_pages > kMaxCount ||
      q->max_pages * c->page_size > kMaxCount)
    return QG_E_SHAPE;
  if (q->reserved != 0) return QG_E_ARG;
  if (q->n_seq > 0 && (!q->starts || !q->lens || (q->max_pages > 0 && !q->tables))) return QG_E_NULL;
  return QG_OK;
}

}  // namespace qgemv_kv

extern "C" {

int qgemv_rope_freqs(int32_t n_rot, double base, int32_t scaling, double factor, double trained, double fast,
                     double slow, double *freqs, double *mscale) {
  if (!freqs) return QG_E_NULL;
  if (scaling < QG_ROPE_NONE || scaling > QG_ROPE_YARN) return QG_E_FMT;
  if (n_rot < 2 || n_rot % 2 != 0 || n_rot > 2 * kAngles) return QG_E_SHAPE;
  if (!std::isfinite(base) || base <= 1.0) return QG_E_ARG;
  if (scaling != QG_ROPE_NONE && (!std::isfinite(factor) || factor < 1.0)) return QG_E_ARG;
  if (scaling == QG_ROPE_YARN && (!std::isfinite(trained) || trained < 1.0 || !std::isfinite(fast) ||
                                  !std::isfinite(slow) || slow <= 0.0 || fast < slow))
    return QG_E_ARG;
  const int half = n_rot / 2;
  if (scaling == QG_ROPE_NTK && half > 1) base *= std::pow(factor, (double)n_rot / (n_rot - 2));
  double lo = 0.0, hi = 0.0;
  if (scaling == QG_ROPE_YARN) {
    // the index whose pair turns `t` times within the trained length
    const double two_pi = 6.283185307179586476925, span = half / std::log(base);
    lo = std::max(std::floor(span * std::log(trained / (fast * two_pi))), 0.0);
    hi = std::min(std::ceil(span * std::log(trained / (slow * two_pi))), (double)n_rot - 1);
    if (hi <= lo) hi = lo + 0.001;  // (a step)
  }
  for (int i = 0; i < half; ++i) {
    const double f = std::pow(base, -(double)i / half);
    if (scaling == QG_ROPE_LINEAR) {
      freqs[i] = f / factor;
    } else if (scaling == QG_ROPE_YARN) {
      const double keep = 1.0 - std::min(std::max((i - lo) / (hi - lo), 0.0), 1.0);
      freqs[i] = f / factor * (1.0 - keep) + f * keep;
    } else {
      freqs[i] = f;
    }
  }
  if (mscale) *mscale = scaling == QG_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return QG_OK;
}

int qgemv_rope(const qg_heads *x, const int32_t *pos, const qg_rope *rope, const qg_heads *y, int32_t inverse,
               qg_stream_t stream) {
  int rc;
  if ((rc = check_heads(x, false, 65536)) || (rc = check_heads(y, true, 65536)) ||
      (rc = check_rope(rope, x->head_dim)))
    return rc;
  if (y->n_tok != x->n_tok || y->n_head != x->n_head || y->head_dim != x->head_dim) return QG_E_SHAPE;
  if (x->n_tok == 0) return QG_OK;
  if (!pos) return QG_E_NULL;
  const bool same = x->data == y->data;
  if (same && (x->type != y->type || x->tok_stride != y->tok_stride || x->head_stride != y->head_stride))
    return QG_E_ARG;
  RopeArgs a = {};
  a.x = heads_of(x);
  a.y = heads_of(y);
  a.turn = turn_of(rope, inverse != 0);
  a.pos = pos;
  a.n_tok = (int)x->n_tok;
  a.n_head = x->n_head;
  // turned in place, the values behind the pairs stay
  a.dim = same ? rope->n_rot : x->head_dim;
  const int pairs = pairs_of(a.turn.half);
  a.units = a.turn.half / pairs + (a.dim - rope->n_rot + 2 * pairs - 1) / (2 * pairs);
  dim3 grid;
  share(x->n_tok, a.n_head, a.units, a.turn.half, a.toks, a.heads, grid);
  in_grids(grid, [&](int64_t first, dim3 part) {
#define QG_RUN(kernel) hipLaunchKernelGGL(kernel, part, dim3(256), 0, stream, a, first)
    QG_KV_PICK(rope_kernel, x->type, pairs, QG_RUN);
#undef QG_RUN
  });
  KV_HIP(hipGetLastError());
  return QG_OK;
}

int qgemv_kv_append(const qg_heads *k, const qg_heads *v, const qg_kv_seqs *seqs, const qg_kv_cache *cache,
                    int32_t layer, const qg_rope *rope, const int32_t *pos, const qg_heads *q, const qg_heads *q_out,
                    qg_stream_t stream) {
  int rc;
  if ((rc = check_cache(cache)) || (rc = check_seqs(seqs, cache)) ||
      (rc = check_heads(k, false, QG_MAX_HEAD_DIM)) || (rc = check_heads(v, false, QG_MAX_HEAD_DIM)) ||
      (rope && (rc = check_rope(rope, cache->head_dim))))
    return rc;
  if (q && ((rc = check_heads(q, false, QG_MAX_HEAD_DIM)) || (rc = check_heads(q_out, true, QG_MAX_HEAD_DIM))))
    return rc;
  if (k->type != v->type || (q && q->type != k->type)) return QG_E_FMT;
  if (k->n_head != cache->n_head || v->n_head != cache->n_head || k->head_dim != cache->head_dim ||
      v->head_dim != cache->head_dim || v->n_tok != k->n_tok)
    return QG_E_SHAPE;
  if (layer < 0 || layer >= cache->n_layer) return QG_E_RANGE;
  if (q) {
    if (!rope) return QG_E_ARG;
    if (q->n_tok != k->n_tok || q->head_dim != k->head_dim || q_out->n_tok != q->n_tok ||
        q_out->n_head != q->n_head || q_out->head_dim != q->head_dim)
      return QG_E_SHAPE;
    if (q_out->data == q->data &&
        (q_out->type != q->type || q_out->tok_stride != q->tok_stride || q_out->head_stride != q->head_stride))
      return QG_E_ARG;
  } else if (q_out) {
    return QG_E_ARG;
  }
  if (k->n_tok == 0 || seqs->n_seq == 0) return QG_OK;
  AppendArgs a = {};
  a.k = heads_of(k);
  a.v = heads_of(v);
  if (q) {
    a.q = heads_of(q);
    a.q_out = heads_of(q_out);
    a.q_heads = q->n_head;
  }
  a.turn = turn_of(rope, 0);
  a.seqs = seqs_of(seqs, cache);
  a.pos = pos;
  a.ck = (uint8_t *)cache->k + layer * cache->layer_stride * 2;
  a.cv = (uint8_t *)cache->v + layer * cache->layer_stride * 2;
  a.page_stride = cache->page_stride;
  a.head_stride = cache->head_stride;
  a.slot_stride = cache->slot_stride;
  a.n_pages = cache->n_pages;
  a.cache_type = cache->type;
  a.n_tok = (int)k->n_tok;
  a.kv_heads = cache->n_head;
  a.dim = cache->head_dim;
  const int pairs = pairs_of(a.turn.half);
  const int turned = a.turn.half / pairs + (a.dim - 2 * a.turn.half + 2 * pairs - 1) / (2 * pairs);
  a.units = std::max(turned, (a.dim + 2 * pairs - 1) / (2 * pairs));
  dim3 grid;
  share(k->n_tok, a.q_heads + 2 * a.kv_heads, a.units, a.turn.half, a.toks, a.heads, grid);
  in_grids(grid, [&](int64_t first, dim3 part) {
#define QG_RUN(kernel) hipLaunchKernelGGL(kernel, part, dim3(256), 0, stream, a, first)
    QG_KV_PICK(append_kernel, k->type, pairs, QG_RUN);
#undef QG_RUN
  });
  KV_HIP(hipGetLastError());
  return QG_OK;
}

}  // extern "C"
