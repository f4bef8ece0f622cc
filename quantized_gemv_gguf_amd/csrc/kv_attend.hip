// kv_attend.hip -- the C ABI of qgemv_kv_attend: checks, the workspace, the shape of a call.
#include "kv_attend.h"

#include <algorithm>
#include <cmath>

using namespace qgemv_kv;

namespace {

// Workgroups of few rows that the compute units hold at once, by their LDS.
int64_t few_at_once(int dim) {
  const int64_t waves = dim <= 128 ? 4 : 2, lds = waves * 2 * 2 * 32 * dim * 2 + 1024;
  return 256 * std::min<int64_t>(163840 / lds, 4);
}

AttendShape shape_of(const qg_heads *q, const qg_kv_seqs *seqs, const qg_kv_cache *cache) {
  AttendShape s = {};
  const int64_t group = q->n_head / cache->n_head, n_seq = seqs->n_seq;
  // (About 16 rows a sequence, on average, the two take about the same: few and
  // many, of 16 rows, 42 and 37 us for 8 sequences of 4000, 32 heads over 8 of 128,
  // bf16; 142 and 150 for 64 heads of 96, fp16; 18 and 29 for one sequence of 8000;
  // of 20 rows 50 and 37, of 17 166 and 150, of 20 19 and 29; of 64 65 and 42.
  // A chunk beside single tokens takes one kernel with them: 63 tokens over up to
  // 2049 positions and 512 over 4096, 64 heads of 96, 595 us, in two calls 411; of
  // 64 heads over 8 of 64 and up to 8192 153 and 174.)
  s.rows = q->n_tok * group > kFewRows * n_seq ? kManyRows : kFewRows;
  const bool few = s.rows == kFewRows;
  // every sequence may end in a partial tile, of one row at least
  s.tiles = std::min(q->n_tok * group, q->n_tok * group / s.rows + n_seq);
  // Parts to cut the keys into: of one sequence as many as run at once, of
  // several, whose parts are not alike, half as many again.
  int64_t parts = few ? few_at_once(cache->head_dim) * (n_seq > 1 ? 3 : 2) / 2 : 512;
  // Enough tiles, or keys for one part: nothing is cut.  (256 tiles of many rows
  // leave room for as many again, which pays for long keys only: 2000 new tokens
  // of 2000, 32 heads over 8 of 128, 53 us, cut 63; 4000 of 4000, 8 heads, 83 and 70.)
  const int64_t least = (q->n_tok * group + s.rows - 1) / s.rows * cache->n_head;
  const int64_t most_keys = seqs->max_pages * cache->page_size;
  const bool whole = few ? least >= parts || most_keys <= kFewPiece
                         : least >= parts || most_keys <= 8 * kManyPiece || (least >= parts / 2 && most_keys <= 2048);
  s.target = whole ? 0 : (int)((parts + cache->n_head - 1) / cache->n_head);
  s.parts = s.tiles + s.target;
  return s;
}

int64_t part_rows_of(const AttendShape &s, const qg_kv_cache *cache) {
  return s.target > 0 && s.tiles > 0 ? s.parts * cache->n_head * s.rows : 0;
}

int check_attend(const qg_heads *q, const qg_kv_seqs *seqs, const qg_kv_cache *cache, bool sizes_only) {
  if (!q || !seqs || !cache) return QG_E_NULL;
  qg_heads h = *q;
  qg_kv_seqs s = *seqs;
  qg_kv_cache c = *cache;
  if (sizes_only) {  // any addresses
    static char some[16] __attribute__((aligned(16)));
    h.data = c.k = c.v = some;
    s.starts = s.lens = s.tables = (const int32_t *)some;
  }
  int rc;
  if ((rc = check_cache(&c)) || (rc = check_seqs(&s, &c)) || (rc = check_heads(&h, false, QG_MAX_HEAD_DIM))) return rc;
  if (h.head_dim != c.head_dim || h.n_head % c.n_head != 0 || h.n_tok * h.n_head > kMaxCount) return QG_E_SHAPE;
  return QG_OK;
}

}  // namespace

extern "C" {

int64_t qgemv_kv_attend_bytes(const qg_heads *q, const qg_kv_seqs *seqs, const qg_kv_cache *cache) {
  const int rc = check_attend(q, seqs, cache, true);
  if (rc) return rc;
  const AttendShape s = shape_of(q, seqs, cache);
  return part_rows_of(s, cache) * (cache->head_dim + 2) * 4;
}

int qgemv_kv_attend(const qg_heads *q, const qg_kv_seqs *seqs, const qg_kv_cache *cache, int32_t layer,
                    const qg_heads *out, float scale, int32_t causal, int32_t window, const float *sinks, float *lse,
                    void *work, int64_t work_bytes, qg_stream_t stream) {
  int rc;
  if ((rc = check_attend(q, seqs, cache, false)) || (rc = check_heads(out, true, QG_MAX_HEAD_DIM))) return rc;
  if (out->n_tok != q->n_tok || out->n_head != q->n_head || out->head_dim != q->head_dim) return QG_E_SHAPE;
  if (layer < 0 || layer >= cache->n_layer) return QG_E_RANGE;
  if (!std::isfinite(scale * kLog2e) || scale <= 0.0f || window < 0) return QG_E_ARG;
  const AttendShape s = shape_of(q, seqs, cache);
  const int64_t part_rows = part_rows_of(s, cache), bytes = part_rows * (cache->head_dim + 2) * 4;
  if (work_bytes < bytes) return QG_E_SIZE;
  if (q->n_tok == 0 || seqs->n_seq == 0) return QG_OK;
  if (bytes > 0 && !work) return QG_E_NULL;
  if ((uintptr_t)work & 15) return QG_E_ARG;
  AttendArgs a = {};
  a.q = heads_of(q);
  a.out = heads_of(out);
  a.k = (const uint16_t *)cache->k + layer * cache->layer_stride;
  a.v = (const uint16_t *)cache->v + layer * cache->layer_stride;
  a.page_stride = cache->page_stride;
  a.head_stride = cache->head_stride;
  a.slot_stride = cache->slot_stride;
  a.seqs = seqs_of(seqs, cache);
  a.sinks = sinks;
  a.lse = lse;
  a.part = (float *)work;
  a.part_rows = part_rows;
  a.n_tok = (int)q->n_tok;
  a.group = q->n_head / cache->n_head;
  a.kv_heads = cache->n_head;
  a.n_pages = (int)cache->n_pages;
  a.scale = scale * kLog2e;
  a.causal = causal != 0;
  a.window = window;
  a.target = s.target;
  const bool wide = q->type != cache->type || out->type != cache->type;
  const auto run = cache->type == QG_F16 ? launch_attend<QG_F16> : launch_attend<QG_BF16>;
  KV_HIP(run(a, s, cache->head_dim, wide, stream));
  return QG_OK;
}

}  // extern "C"
