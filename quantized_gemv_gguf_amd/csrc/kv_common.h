// kv_common.h -- what the sources of include/qgemv_kv.h share: element types,
// small wave helpers, the arguments of heads, caches and sequences.
#pragma once

#include <hip/hip_runtime.h>

#include "qgemv_kv.h"

namespace qgemv_detail {
int record_hip_error(hipError_t e, const char *what);  // qgemv.hip: for qgemv_last_hip_error
}

#define KV_HIP(call)                                                       \
  do {                                                                     \
    hipError_t e_ = (call);                                                \
    if (e_ != hipSuccess) return qgemv_detail::record_hip_error(e_, #call); \
  } while (0)

namespace qgemv_kv {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <int T> struct Elem;
template <> struct Elem<QG_F32> { typedef float Raw; };
template <> struct Elem<QG_F16> { typedef _Float16 Raw; };
template <> struct Elem<QG_BF16> { typedef __bf16 Raw; };

// N values from / to any element-aligned address, as one access of N elements.
template <int T, int N>
__device__ __forceinline__ void load_n(const void *p, float (&v)[N]) {
  typedef typename Elem<T>::Raw V __attribute__((ext_vector_type(N)));
  V r;
  __builtin_memcpy(&r, p, N * sizeof(typename Elem<T>::Raw));
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (float)r[i];
}
template <int T, int N>
__device__ __forceinline__ void store_n(void *p, const float (&v)[N]) {
  typedef typename Elem<T>::Raw V __attribute__((ext_vector_type(N)));
  V r;
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = (typename Elem<T>::Raw)v[i];
  __builtin_memcpy(p, &r, N * sizeof(typename Elem<T>::Raw));
}

// The same with the type known at run time only (uniform: one branch).
template <int N> __device__ __forceinline__ void load_as(int type, const uint8_t *p, int64_t at, float (&v)[N]) {
  if (type == QG_F32) load_n<QG_F32>(p + at * 4, v);
  else if (type == QG_F16) load_n<QG_F16>(p + at * 2, v);
  else load_n<QG_BF16>(p + at * 2, v);
}
template <int N> __device__ __forceinline__ void store_as(int type, uint8_t *p, int64_t at, const float (&v)[N]) {
  if (type == QG_F32) store_n<QG_F32>(p + at * 4, v);
  else if (type == QG_F16) store_n<QG_F16>(p + at * 2, v);
  else store_n<QG_BF16>(p + at * 2, v);
}

__host__ __device__ inline int elem_size(int type) {
  return type == QG_F32 ? 4 : type == QG_F16 || type == QG_BF16 ? 2 : 0;
}

// The device's view of a qg_heads and of a qg_kv_seqs.
struct Heads {
  uint8_t *p;
  int64_t tok_stride, head_stride;
  int type;
};
struct Seqs {
  const int32_t *starts, *lens, *tables;
  int64_t max_pages;
  int n_seq, page_shift;
};

// The row range of sequence s, kept within the activations' rows whatever the
// arrays hold, and its length (which its table need not hold).
__device__ __forceinline__ void seq_rows(const Seqs &q, int s, int n_tok, int &start, int &n, int &len) {
  start = min(max(q.starts[s], 0), n_tok);
  n = min(max(q.starts[s + 1], start), n_tok) - start;
  len = max(q.lens[s], 0);
}
// Positions that a table holds.
__device__ __forceinline__ int room_of(const Seqs &q) { return (int)(q.max_pages << q.page_shift); }

constexpr int64_t kMaxCount = 0x7fff0000;  // tokens, pages, positions: an index a little past the end stays an int

// Workgroups of one launch in x: at most 2^31 threads.
constexpr int64_t kMaxGrid = 1 << 23;

// kv.hip: statuses of the arguments.
int check_heads(const qg_heads *h, bool out, int64_t most_dim);
int check_cache(const qg_kv_cache *c);
int check_seqs(const qg_kv_seqs *q, const qg_kv_cache *c);

__host__ __device__ constexpr int log2_of(int64_t v) {
  int n = 0;
  while ((1ll << n) < v) ++n;
  return n;
}

inline Heads heads_of(const qg_heads *h) {
  return {(uint8_t *)h->data, h->tok_stride, h->head_stride, h->type};
}
inline Seqs seqs_of(const qg_kv_seqs *q, const qg_kv_cache *c) {
  return {q->starts, q->lens, q->tables, q->max_pages, q->n_seq, log2_of(c->page_size)};
}

}  // namespace qgemv_kv
