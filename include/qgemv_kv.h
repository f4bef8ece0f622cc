/*
 * qgemv_kv.h -- a paged cache of keys and values on an AMD Instinct MI355X
 * (gfx950): rotary positions, new tokens written into the cache, their
 * attention over it, and the bookkeeping of its pages.
 * Part of libqgemv.so; qgemv.h holds the status codes and the conventions,
 * qgemv_mx.h the float types; both hold here too (host-side validation before
 * any HIP call, a refused call enqueues nothing and leaves every output
 * untouched, caller's memory and stream, no waiting, no allocation, safe under
 * stream capture).  The caller's current device must be the buffers' and the
 * stream's device.  Calls that write nothing in common may run at once.
 *
 * What a decoder layer does between its QKV product and its output product
 * (RAMforge README, "Milestone 5", and neurostream README, "How it works",
 * leave it to their models), for one token of each of many sequences or for
 * chunks of prompts:
 *
 *     qgemv_kv_resize(pool, cache, lens)            once a step: room for the new tokens
 *     qgemv_kv_append(k, v, seqs, cache, q, q_out)  a layer: positions, keys and values stored
 *     qgemv_kv_attend(q_out, seqs, cache, out)      a layer: softmax(q k^T) v
 *
 * with qgemv_kv_fork where sequences share what they have in common (a prompt,
 * a beam's past) and qgemv_kv_compact where pages are to be given back.  Every
 * length, page and place stays on the device.
 *
 * Outputs of one call do not depend on timing, the stream or earlier calls: no
 * kernel uses floating-point atomics, and what integer atomics count does not
 * depend on their order.
 */
#ifndef QGEMV_KV_H
#define QGEMV_KV_H

#include "qgemv_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most sequences of one call, and most query heads. */
#define QG_MAX_SEQS 4096
#define QG_MAX_HEADS 1024
/* Largest head of the cache: a multiple of 32, the inputs of one matrix instruction. */
#define QG_MAX_HEAD_DIM 256

/* Heads of tokens in device memory: head h of token t starts at element
 * t * tok_stride + h * head_stride of data, its head_dim elements contiguous
 * (a slice of a QKV product's rows has the product's row length as tok_stride).
 * data aligned to one element; strides >= 0, an output's heads may not overlap
 * (QG_E_ARG).  Inputs and outputs of one call must not overlap, but where it
 * says so. */
typedef struct qg_heads {
  void *data;
  int32_t type;     /* enum qg_float */
  int32_t reserved; /* must be 0 */
  int64_t n_tok;    /* 0 .. 2^31 - 2^16 */
  int32_t n_head;   /* 1 .. QG_MAX_HEADS */
  int32_t head_dim;
  int64_t tok_stride;
  int64_t head_stride;
} qg_heads;

enum qg_rope_scaling { QG_ROPE_NONE = 0, QG_ROPE_LINEAR = 1, QG_ROPE_NTK = 2, QG_ROPE_YARN = 3 };

/* Rotary positions: of each head's first n_rot values, pair i is turned by
 * position * freqs[i] and multiplied by mscale; the values behind stay.
 * Pair i is (i, i + n_rot / 2), or (2 i, 2 i + 1) where interleaved. */
typedef struct qg_rope {
  const double *freqs; /* device, n_rot / 2 values: radians a position */
  int32_t n_rot;       /* even, 2 .. head_dim */
  int32_t interleaved; /* 0 or 1 */
  double mscale;       /* factor of the turned values, finite */
} qg_rope;

/* The keys and values of every layer.  Element (layer, page, head, slot, i) is
 * at layer * layer_stride + page * page_stride + head * head_stride + slot *
 * slot_stride + i, of k and of v alike.  Both 16-byte aligned, strides
 * multiples of 8 elements, positive, and such that no two elements meet
 * (QG_E_ARG): any order of the axes.  A page's keys in a layer are at most 2^33
 * elements. */
typedef struct qg_kv_cache {
  void *k;
  void *v;
  int32_t type;      /* QG_F16 or QG_BF16 */
  int32_t page_size; /* slots of a page: a power of two up to 65536 */
  int32_t n_layer;
  int32_t n_head;    /* 1 .. QG_MAX_HEADS */
  int32_t head_dim;  /* a multiple of 32 up to QG_MAX_HEAD_DIM */
  int32_t reserved;  /* must be 0 */
  int64_t n_pages;   /* 1 .. 2^31 - 2^16 */
  int64_t layer_stride, page_stride, head_stride, slot_stride;
} qg_kv_cache;

/* The sequences of a call, all device arrays.  Position p of sequence s lies
 * in slot p % page_size of page tables[s * max_pages + p / page_size].  Of its
 * lens[s] positions the last starts[s + 1] - starts[s] are its new tokens:
 * rows starts[s] and following of the activations.  A page outside [0,
 * n_pages) is not there: nothing is written to it, and its positions are as
 * masked (so the pages a sliding window has passed may be given back).  So
 * are positions below 0 and from max_pages * page_size.  starts rises from 0 on; rows behind the
 * last sequence belong to none. */
typedef struct qg_kv_seqs {
  const int32_t *starts; /* n_seq + 1 */
  const int32_t *lens;   /* n_seq */
  const int32_t *tables; /* n_seq x max_pages */
  int32_t n_seq;         /* 0 .. QG_MAX_SEQS */
  int32_t reserved;      /* must be 0 */
  int64_t max_pages;     /* 0 .., max_pages * page_size at most 2^31 - 2^16 */
} qg_kv_seqs;

/* Who holds which page; device memory that the calls below keep up to date.
 * A sequence's entries are in use up to its length and -1 behind; refs counts
 * the sequences that hold a page, used has a bit (page % 32 of word page / 32)
 * for every page that any holds.  tables -1 and the rest 0 is an empty pool.
 * lens and tables may serve as a qg_kv_seqs'.  One call at a time may use a
 * pool. */
typedef struct qg_kv_pool {
  int32_t *tables; /* n_seq x max_pages */
  int32_t *lens;   /* n_seq */
  int32_t *refs;   /* n_pages */
  int32_t *used;   /* (n_pages + 31) / 32 */
  int32_t n_seq;   /* 1 .. QG_MAX_SEQS */
  int32_t page_size;
  int64_t max_pages; /* 1 .., max_pages * page_size at most 2^31 - 2^16,
                        n_seq * max_pages below 2^31 */
  int64_t n_pages;   /* 1 .. QG_MAX_POOL_PAGES */
  void *work;        /* device, 16-byte aligned; holds nothing between calls */
  int64_t work_bytes;
} qg_kv_pool;

#define QG_MAX_POOL_PAGES (1 << 22)

/* Writes the n_rot / 2 frequencies of rotary positions of this base to host
 * memory, and to *mscale (may be NULL) the factor that belongs to them:
 *   NONE    base^(-2 i / n_rot), 1
 *   LINEAR  the same over `factor`: positions interpolated
 *   NTK     the base times factor^(n_rot / (n_rot - 2)): the slowest pair turns
 *           `factor` times slower, the fastest as before
 *   YARN    pairs that turn at least `fast` times within the `trained` length
 *           as NONE, those that turn at most `slow` times as LINEAR, in between
 *           a mixture by the pair's index between whole numbers (the border
 *           indices rounded down and up and kept within [0, n_rot - 1]); mscale
 *           = 0.1 ln(factor) + 1
 * n_rot even and >= 2, base > 1, factor >= 1, trained >= 1, fast >= slow > 0,
 * all finite (those the scaling does not use are not looked at). */
int qgemv_rope_freqs(int32_t n_rot, double base, int32_t scaling, double factor, double trained, double fast,
                     double slow, double *freqs, double *mscale);

/* y[t] = x[t] turned by position pos[t] (device, n_tok), or with inverse != 0 by
 * -pos[t]: the gradient of the turn (dx from dy; mscale applies again).  Angles
 * are reduced in 64 bits, the turn is in fp32, y is rounded once.  y has x's
 * sizes, any float type; y may be x itself (same address, type and strides),
 * otherwise they must not overlap.  head_dim 1 .. 2^16 here, n_rot up to 1024. */
int qgemv_rope(const qg_heads *x, const int32_t *pos, const qg_rope *rope, const qg_heads *y, int32_t inverse,
               qg_stream_t stream);

/* Stores the new tokens' keys (turned by rope, as they are where it is NULL) and
 * values (as they are) in `layer` of the cache, each value rounded once to its
 * type; and, where q is not NULL, turns their queries into q_out in the same
 * launch.  k, v and q share one type; k and v have the cache's heads.  A token's
 * position is pos[row] (device, n_tok) for the turn, or where pos is NULL the
 * one that it is stored at.  Rows that belong to no sequence are left as they
 * were in q_out too.  Where sequences share a page, only one may append to it
 * (qgemv_kv_resize sees to that).  Without rope q must be NULL. */
int qgemv_kv_append(const qg_heads *k, const qg_heads *v, const qg_kv_seqs *seqs, const qg_kv_cache *cache,
                    int32_t layer, const qg_rope *rope, const int32_t *pos, const qg_heads *q, const qg_heads *q_out,
                    qg_stream_t stream);

/* Attention of the new tokens over their sequences' positions in `layer`: row t,
 * at position p = lens[s] - (starts[s + 1] - t) of its sequence, head h of q
 * with head h / (q heads / cache heads) of the cache,
 *     s_j = scale <q[t, h], k_j>     for the positions j that t sees,
 *     out[t, h] = sum_j exp(s_j - m) v_j / (sum_j exp(s_j - m) + exp(sinks[h] - m)).
 * It sees j < lens[s] whose page is there, with causal != 0 j <= p only, with
 * window > 0 j > p - window only.  What is in masked places (infinities, NaN)
 * does not matter.  sinks (device, one fp32 per q head: a logit without a value)
 * and lse (device, n_tok x q heads, fp32: the log of the denominator, m's factor
 * put back) may be NULL.  A row that sees nothing, or whose scores are all -inf,
 * gets zeros, whatever its values hold, and lse the sink's logit or -inf.  A row
 * that sees a value without a size (infinite, NaN) has none there either: NaN, or
 * the infinity where its weight is not 0 (one too small for its type may be).  An
 * infinite q or key may make a score NaN, and so the row, where q is taken in terms.
 * Rows that belong to no sequence are left as they were.
 * Scores, sums and the softmax are fp32.  Where q and out have the cache's type,
 * the weights exp(s_j - m) are rounded once to it before they meet v (as the
 * matrix cores take them), 2^-11 or 2^-8 of each; otherwise q and the weights are
 * taken in two terms of QG_F16, 2^-22 of each, or three of QG_BF16, 2^-24.  What
 * is far below the largest adds nothing: weights are held to 2^-32 of the row's
 * largest at least in QG_F16, 2^-118 in QG_BF16, q's terms to 2^-39 of the row's
 * largest value in QG_F16, in QG_BF16 to 2^-133.
 * out is rounded once.  The order of sums may differ for another number of rows
 * or sequences and other lengths of the others.  One of two kernels serves all of
 * a call, by its rows a sequence on average: single tokens and long chunks can be
 * faster in calls of their own.
 * scale > 0, up to 2^127; window >= 0; out has q's sizes; q heads a multiple of
 * the cache's heads, n_tok * q heads at most 2^31 - 2^16.  work: device, 16-byte aligned, at least
 * qgemv_kv_attend_bytes, holds nothing between calls; calls that may run at
 * once need one each (QG_E_SIZE where it is too small). */
int qgemv_kv_attend(const qg_heads *q, const qg_kv_seqs *seqs, const qg_kv_cache *cache, int32_t layer,
                    const qg_heads *out, float scale, int32_t causal, int32_t window, const float *sinks, float *lse,
                    void *work, int64_t work_bytes, qg_stream_t stream);

/* Bytes of the workspace of a qgemv_kv_attend call with these sizes (pointers
 * are not looked at), or a negative status.  A call with fewer tokens, sequences
 * or heads may need more than a larger one, whose keys are cut into fewer parts
 * (with tables for 32768 positions, 32 heads over 8 of 128, one sequence of 2048
 * tokens needs none and of 8 tokens 35 MB): a workspace for several kinds of calls
 * is as large as the largest of their sizes. */
int64_t qgemv_kv_attend_bytes(const qg_heads *q, const qg_kv_seqs *seqs, const qg_kv_cache *cache);

/* Bytes of a pool's workspace, or a negative status. */
int64_t qgemv_kv_pool_bytes(int64_t n_seq, int64_t max_pages, int64_t n_pages);

/* Cuts and grows every sequence s to lens[s] positions (device, n_seq; a
 * negative one leaves it as it is, 0 lets it go).  First the pages that are no
 * longer needed are let go.  Then, sequence after sequence, growing ones take
 * the free pages of the lowest numbers.  A last page that is partly filled and
 * held by others too is copied, in every layer, to a page of the sequence's own
 * before it grows into it; where all who hold it are to grow, the first of them
 * keeps it.  A sequence whose pages, with those of all before it, are not there any
 * more or that would pass max_pages stays at its old length (pool->lens tells), and
 * so does one that would keep a page with a longer sequence that stays.
 * The cache's page_size and n_pages must be the pool's (QG_E_SHAPE). */
int qgemv_kv_resize(const qg_kv_pool *pool, const qg_kv_cache *cache, const int32_t *lens, qg_stream_t stream);

/* All at once, every sequence s becomes what sequence from[s] was (device,
 * n_seq; s itself: stays), sharing its pages: forks, reordered beams.  -1 lets s
 * go; another id outside [0, n_seq) leaves it as it is. */
int qgemv_kv_fork(const qg_kv_pool *pool, const int32_t *from, qg_stream_t stream);

/* Moves the pages in use to the lowest numbers, their order kept among those
 * that move: the i-th page in use from the number of used pages on goes to the
 * i-th free one below it, in every layer. */
int qgemv_kv_compact(const qg_kv_pool *pool, const qg_kv_cache *cache, qg_stream_t stream);

/* Copies page src[i] to page dst[i] (device, n each) in every layer.  A pair
 * with an id outside [0, n_pages) does nothing.  A page may be a source many
 * times; it may be a destination once, and then no source (its content would
 * depend on timing). */
int qgemv_kv_copy(const qg_kv_cache *cache, const int32_t *src, const int32_t *dst, int64_t n, qg_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QGEMV_KV_H */
