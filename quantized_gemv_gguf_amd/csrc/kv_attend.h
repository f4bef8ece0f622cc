// kv_attend.h -- attention of new tokens over a paged cache.
//
// A row (t, h) of q with the keys it sees, any m near max_j s_j, gives
//     o = sum_j e^(s_j - m) v_j / l,   l = sum_j e^(s_j - m) + e^(sink - m).
// Keys are walked once, in pieces: of a piece's m', sum l' and products
// o' (all fp32) the running ones become m'' = max(m, m'), l'' = l e^(m - m'') +
// l' e^(m' - m''), and o'' likewise; so do those of parts of the keys that
// different workgroups have walked.
//
// Matrix instructions take S^T = K Q^T with the keys as rows and the q rows as
// columns.  A lane then holds several keys' scores of one q row, which is the
// layout that O^T = V^T P^T takes P^T in: weights go from scores to products
// within a lane's registers, a row's maximum and factor are one value a lane.
// (The keys of a product may come in any order, if v's do too.)
//
// The q heads that share a head of the cache are rows of one tile: of sequence
// s, row r is token r / group, head r % group.
#pragma once

#include "kv_common.h"

namespace qgemv_kv {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

struct AttendArgs {
  Heads q, out;
  const uint16_t *k, *v;  // the layer's
  int64_t page_stride, head_stride, slot_stride;
  Seqs seqs;
  const float *sinks;
  float *lse;
  float *part;  // of parts: rows of dim sums, then rows of (m, l)
  int64_t part_rows;
  int n_tok, group, kv_heads, n_pages;
  float scale;  // log2(e) times the caller's
  int causal, window;
  int target;  // parts to cut the keys into, at most, beyond one a tile; 0: no cuts
};

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2f_of(float x) { return __builtin_amdgcn_logf(x); }
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_huge_valf();

// ---------------------------------------------------------------------------
// Which workgroup takes what.  Lengths are on the device, so each finds its
// tile of rows and part of the keys itself: pieces of kPiece keys are counted
// over all tiles, and a sequence's tiles are cut into parts of so many pieces
// that about `target` parts come out in all.  A wave does this for itself, its
// lanes over the sequences: no barrier.
// ---------------------------------------------------------------------------

constexpr int kFewRows = 16, kFewPiece = 128;

// The first position that one at pos sees, and the end of those that it sees,
// of a sequence of this length, within its table.
__device__ __forceinline__ int first_seen(const AttendArgs &a, int pos) {
  return a.window ? (int)max((int64_t)pos - a.window + 1, (int64_t)0) : 0;
}
__device__ __forceinline__ int end_seen(const AttendArgs &a, int pos, int len) {
  return min(a.causal ? pos + 1 : len, room_of(a.seqs));
}

struct Item {
  int s, tile, part, parts;  // parts: of this tile; 0: nothing to do
  int first;                 // the tile's first part among all parts
  int start, n, len;         // the sequence's rows and length
};

template <int ROWS, int PIECE> struct Plan {
  const AttendArgs &a;
  __device__ Plan(const AttendArgs &args) : a(args) {}

  // Tiles of a sequence and the pieces of keys that its rows see.
  __device__ void size_of(int s, int &tiles, int &pieces) const {
    int start, n, len;
    seq_rows(a.seqs, s, a.n_tok, start, n, len);
    tiles = (int)(((int64_t)n * a.group + ROWS - 1) / ROWS);
    const int hi = end_seen(a, len - 1, len), lo = min(first_seen(a, len - n), hi);
    pieces = max(1, (int)(((int64_t)hi - lo + PIECE - 1) / PIECE));
  }
  // Pieces of a part.  One of many rows costs its sums' way through memory, as
  // much as some pieces' products: it gets eight at least (100 new tokens of each
  // of 4 sequences up to 4000, 32 heads over 8 of 128: 30 us, with sixteen 36).
  __device__ int pieces_each(int64_t all) const {
    return max((int)((all + a.target - 1) / a.target), ROWS == kFewRows ? 1 : 8);
  }
  // The item of this number among parts (BY_TILE: among tiles).
  template <bool BY_TILE> __device__ Item find(int number) const {
    const int lane = threadIdx.x & 63, n_seq = a.seqs.n_seq;
    if (n_seq == 1) {  // (the same without a scan: 1.1 us less of a launch's start)
      int tiles, pieces;
      size_of(0, tiles, pieces);
      const int parts = a.target > 0 ? (pieces - 1) / pieces_each((int64_t)tiles * pieces) + 1 : 1;
      const int tile = BY_TILE ? number : number / parts;
      Item it = {};
      if (tile >= tiles) return it;
      it.parts = parts;
      it.part = BY_TILE ? 0 : number - tile * parts;
      it.first = tile * parts;
      it.tile = tiles - 1 - tile;
      seq_rows(a.seqs, 0, a.n_tok, it.start, it.n, it.len);
      return it;
    }
    int each = 0x7fffffff;  // pieces of a part
    if (a.target > 0) {
      int64_t all = 0;
      for (int s0 = 0; s0 < n_seq; s0 += 64) {
        int tiles = 0, pieces = 0;
        if (s0 + lane < n_seq) size_of(s0 + lane, tiles, pieces);
        all += (int64_t)tiles * pieces;
      }
#pragma unroll
      for (int d = 32; d > 0; d /= 2) all += __shfl_xor(all, d);
      each = pieces_each(all);
    }
    Item it = {};
    int items = 0, parts_before = 0;  // of the sequences before s0
    for (int s0 = 0; s0 < n_seq; s0 += 64) {
      int tiles = 0, pieces = 1;
      if (s0 + lane < n_seq) size_of(s0 + lane, tiles, pieces);
      const int parts = a.target > 0 ? (pieces - 1) / each + 1 : 1;
      int sum = BY_TILE ? tiles : tiles * parts, sum_parts = tiles * parts;
      const int mine = sum, mine_parts = sum_parts;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(sum, d), p = __shfl_up(sum_parts, d);
        if (lane >= d) {
          sum += o;
          sum_parts += p;
        }
      }
      const uint64_t here = __ballot(items + sum > number);
      if (here) {
        const int l = __builtin_ctzll(here);
        const int in = number - items - __builtin_amdgcn_readlane(sum - mine, l);
        const int p = __builtin_amdgcn_readlane(parts, l);
        const int tile = BY_TILE ? in : in / p;
        it.s = s0 + l;
        it.parts = p;
        it.part = BY_TILE ? 0 : in - tile * p;
        it.first = parts_before + __builtin_amdgcn_readlane(sum_parts - mine_parts, l) + tile * p;
        // (the last rows, which see the most, first)
        it.tile = __builtin_amdgcn_readlane(tiles, l) - 1 - tile;
        seq_rows(a.seqs, it.s, a.n_tok, it.start, it.n, it.len);
        return it;
      }
      items += __builtin_amdgcn_readlane(sum, 63);
      parts_before += __builtin_amdgcn_readlane(sum_parts, 63);
    }
    return it;
  }
};

// The keys that a tile's rows see: from the first row's first to the last row's
// last; and those that all of them see.
struct Range {
  int lo, hi, all_lo, all_hi;
};
template <int ROWS> __device__ __forceinline__ Range range_of(const AttendArgs &a, const Item &it) {
  const int first = it.tile * ROWS / a.group;
  const int last = (min(it.n * a.group, (it.tile + 1) * ROWS) - 1) / a.group;
  const int old = it.len - it.n;  // (may be below 0: then the first rows see nothing)
  Range r;
  r.hi = max(end_seen(a, old + last, it.len), 0);
  r.lo = min(first_seen(a, old + first), r.hi);
  r.all_lo = first_seen(a, old + last);
  r.all_hi = end_seen(a, old + first, it.len);
  return r;
}

// ---------------------------------------------------------------------------
// Element types of the cache, and the terms of an fp32 value in them.
// ---------------------------------------------------------------------------

template <int T> struct Kind;
template <> struct Kind<QG_F16> {
  typedef _Float16 H;
  typedef _Float16 V8 __attribute__((ext_vector_type(8)));
  static constexpr int kWide = 2;            // terms that hold an fp32 (22 bits and the sign of the second)
  // log2 of a row's largest weight: of 16 binades above 1 and 24 below, weights
  // of at most 1 would use the lower ones alone, and small ones would lose bits
  // that their sum l counts.  So they are lost below 2^-40 of the largest.
  static constexpr float kTop = 15.0f;
  // and of a q row's that is taken in terms: its values down to 2^-15 of the
  // largest have 22 bits, smaller ones are held to 2^-39 of it
  static constexpr int kRowTop = 14;
  static constexpr uint32_t kExp = 0x7c00u;  // the exponent of infinities and NaN
  static constexpr uint32_t kOne = 0x3c00u;
  static __device__ __forceinline__ f32x4 mfma16(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma32(V8 a, V8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};
template <> struct Kind<QG_BF16> {
  typedef __bf16 H;
  typedef __bf16 V8 __attribute__((ext_vector_type(8)));
  static constexpr int kWide = 3;
  static constexpr float kTop = 0.0f;  // (bf16 has fp32's range, and values as large)
  static constexpr int kRowTop = 0;
  static constexpr uint32_t kExp = 0x7f80u;
  static constexpr uint32_t kOne = 0x3f80u;
  static __device__ __forceinline__ f32x4 mfma16(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma32(V8 a, V8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};

// x as a sum of NT values of the type: each the nearest to what the ones before leave.
template <int T, int NT> __device__ __forceinline__ void terms_of(const float (&x)[8], typename Kind<T>::V8 (&t)[NT]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float left = x[i];
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      t[k][i] = (typename Kind<T>::H)left;
      if (k + 1 < NT) left -= (float)t[k][i];
    }
  }
}

// The same of an fp32 row's values.  bf16's three terms hold all 24 bits (down to
// 2^-133, where bf16 ends: looking for rows that lie below costs prompts with a
// window 2%); the first is cut, not rounded, which would make the largest infinite.
template <int T, int NT> __device__ __forceinline__ void row_terms_of(const float (&x)[8], typename Kind<T>::V8 (&t)[NT]) {
  if (T == QG_BF16 && NT == 3) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float cut = __uint_as_float(__float_as_uint(x[i]) & 0xffff0000u), left = x[i] - cut;
      t[0][i] = (typename Kind<T>::H)cut;
      t[1][i] = (typename Kind<T>::H)left;
      t[NT - 1][i] = (typename Kind<T>::H)(left - (float)t[1][i]);
    }
  } else {
    terms_of<T, NT>(x, t);
  }
}

// The exponent of the largest of a row's values (0 for a row of zeros, infinities
// and NaN): an fp32 row divided by its power of 2 has terms in fp16.
__device__ __forceinline__ int row_exponent(float most) {
  const uint32_t bits = __float_as_uint(most) & 0x7fffffff;
  const int e = (int)(bits >> 23);
  return bits == 0 || e == 255 ? 0 : e > 0 ? e - 127 : -118 - __builtin_clz(bits);
}

// The scale of such a row is scale * 2^e; where that would pass fp32, the scores
// need not: they are multiplied by 2^more first.
struct RowScale {
  float scale;
  int more;
};
__device__ __forceinline__ RowScale row_scale(float scale, int e) {
  const int at = (int)(__float_as_uint(scale) >> 23) - 127;
  const int more = max(at + e - 126, 0);
  return {ldexpf(scale, e - more), more};
}

// Lanes that are 16 and 32 apart hold the same q row: the largest, the sum.
__device__ __forceinline__ float max_of_row16(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float sum_of_row16(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// Two values of the type in a word: are both finite?  Those that are, zeros for the others.
template <int T> __device__ __forceinline__ bool finite2(uint32_t w) {
  constexpr uint32_t e = Kind<T>::kExp;
  return (w & e) != e && (w >> 16 & e) != e;
}
template <int T> __device__ __forceinline__ uint32_t only_finite2(uint32_t w) {
  constexpr uint32_t e = Kind<T>::kExp;
  return ((w & e) == e ? 0 : w & 0xffff) | ((w >> 16 & e) == e ? 0 : w & 0xffff0000u);
}

// The bits from number n on, of 32.
__device__ __forceinline__ uint32_t bits_from(int n) { return n >= 32 ? 0u : ~0u << max(n, 0); }

// Values of v without a size (infinities, NaN) must not reach the rows that may
// not see them: a product with a weight of 0 would be NaN.  Where a tile's rows
// differ in what they see, such values are taken out of the products, and after
// all keys they are counted, kind by kind, with ones in place of the weights of
// the keys a row sees; a count adds the kind itself, which no factor changes.
// (The values are read again from the cache.)
enum Kinds { kNan = 0, kUp = 1, kDown = 2 };
template <int T> __device__ __forceinline__ uint32_t is_kind(uint32_t x, int kind) {
  constexpr uint32_t e = Kind<T>::kExp;
  const bool yes = kind == kNan ? (x & 0x7fff) > e : x == (kind == kUp ? e : e | 0x8000u);
  return yes ? Kind<T>::kOne : 0;
}
__device__ __forceinline__ float of_kind(float count, int kind) {
  return count > 0.0f ? kind == kNan ? __builtin_nanf("") : kind == kUp ? kInf : -kInf : 0.0f;
}

// A finished row's factor (or that no key of its weighs anything: then its sums
// may be NaN, of weights 0 and values without a size, and it is zeros), and the
// logarithm of its denominator (base e).
__device__ __forceinline__ void finish_row(const AttendArgs &a, int head, float m, float l, float &f, bool &none,
                                           float &lse) {
  none = l == 0.0f;
  if (a.sinks) {
    const float z = a.sinks[head] * kLog2e, top = fmaxf(m, z);
    const float w = top == -kInf ? 0.0f : exp2_of(z - top);
    const float keep = m == -kInf ? 0.0f : exp2_of(m - top);
    l = l * keep + w;
    f = keep / l;
    m = top;
  } else {
    f = 1.0f / l;
  }
  lse = l == 0.0f ? -kInf : (m + log2f_of(l)) * kLn2;
}

template <int N> __device__ __forceinline__ void store_row(const Heads &h, int64_t t, int head, int at,
                                                           const float (&v)[N]) {
  store_as(h.type, h.p, t * h.tok_stride + head * h.head_stride + at, v);
}

// Byte offset of a key's row in the cache's head, and whether its page is there.
struct KeyAt {
  int64_t at;
  bool there;
};
__device__ __forceinline__ KeyAt key_at(const AttendArgs &a, int key, int page) {
  const bool there = (unsigned)page < (unsigned)a.n_pages;
  return {((there ? page : 0) * a.page_stride + (key & ((1 << a.seqs.page_shift) - 1)) * a.slot_stride) * 2, there};
}

// One asynchronous copy of 16 bytes a lane to LDS at lds + 16 lane.  The
// compiler's own waits would drain it before any read of LDS; here the kernels
// wait themselves, a tile or more later.
__device__ __forceinline__ void copy_to_lds(const uint8_t *src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void copy_to_lds(const uint8_t *base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
template <int N> __device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// ---------------------------------------------------------------------------
// Few rows: tiles of 16.  Bound by memory: each wave walks every kWaves-th 32
// keys through a ring of its own in LDS, filled by asynchronous copies some
// tiles ahead: no barrier, no registers for what is under way, and lanes next to
// each other copy what lies next to each other.  (Loaded in the layout of the
// matrix instructions, 64 requests an instruction, the next tile in registers:
// 64 sequences up to 8192, 64 heads over 8 of 64, 148 us; so, 114, 5.2 TB/s.
// 131009 positions of 64 heads of 96, fp32 rows: 535, 6.0.)  16 x 16 x 32
// instructions; K^T comes by 16-byte reads, V^T by the transposing 8-byte ones.
// A row of 2 D bytes begins at the same bank as another one, so its 16-byte
// pieces lie at places exchanged by the key's low bits, differently for K and V:
// as the reads that go together fall on different banks.
// ---------------------------------------------------------------------------

template <int D> struct FewTile {
  static constexpr int CH = D / 8;                 // pieces of a row
  static constexpr int kBytes = 32 * D * 2;        // of a tile's k or v
  static constexpr int kWaves = D <= 128 ? 4 : 2;  // of a workgroup
  static constexpr int kDepth = 2;                 // tiles of a ring
  static constexpr int kBanks = D / 2 % 64;        // where the next row begins
  static __host__ __device__ constexpr int k_turn(int key) {
    return kBanks == 0 ? key & 15 : kBanks == 32 ? (key >> 1) & 7 : (key >> 2) & 3;
  }
  static __host__ __device__ constexpr int v_turn(int key) {
    return kBanks == 0 ? (key & 7) << 1 : kBanks == 32 ? ((key >> 1) & 3) << 1 : ((key >> 2) & 1) << 1;
  }
};

template <int T, int D, int NT>
__global__ void __launch_bounds__(64 * FewTile<D>::kWaves) attend_few_kernel(AttendArgs a, int64_t group0) {
  using K = Kind<T>;
  using V8 = typename K::V8;
  using M = FewTile<D>;
  constexpr int E = D / 16, ST = D / 32, CH = M::CH, W = M::kWaves, S = M::kDepth;
  constexpr int kCopies = CH / 4;   // of 16 keys' k, or v
  constexpr int kTileCopies = CH;   // of a tile
  constexpr int kStride = D + 4;    // of a row's sums in LDS: rows in other banks
  constexpr int kRing = W * S * 2 * M::kBytes, kSums = W * kFewRows * kStride * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing > kSums ? kRing : kSums];
  __shared__ float2 stats[W][kFewRows];

  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int number = (int)((group0 + blockIdx.x) / a.kv_heads);
  const int head = (int)(group0 + blockIdx.x - (int64_t)number * a.kv_heads);
  const Item it = Plan<kFewRows, kFewPiece>(a).template find<false>(number);
  if (it.parts == 0) return;
  const Range range = range_of<kFewRows>(a, it);
  // this part's keys: whole pieces from a multiple of 32 on
  const int lo = range.lo & ~31, pieces = max(0, (int)(((int64_t)range.hi - lo + kFewPiece - 1) / kFewPiece));
  const int share = (pieces + it.parts - 1) / it.parts;
  const int begin = lo + min(pieces, it.part * share) * kFewPiece;
  const int end = min(range.hi, lo + min(pieces, (it.part + 1) * share) * kFewPiece);

  const uint8_t *ck = (const uint8_t *)(a.k + head * a.head_stride), *cv = (const uint8_t *)(a.v + head * a.head_stride);
  const int32_t *table = a.seqs.tables + it.s * a.seqs.max_pages;
  const int last_key = max(end - 1, 0);
  constexpr int kStep = 32 * W;
  uint8_t *const ring = lds + wave * S * 2 * M::kBytes;
  const uint32_t ring_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)ring;
  const auto page_of = [&](int key) { return table[min(key, last_key) >> a.seqs.page_shift]; };
  // (the same for a uniform key, through the scalar cache: waiting for a vector
  // load would wait for the copies too, 145 us instead of 117 in the case above)
  const auto page_at = [&](int key) {
    typedef const __attribute__((address_space(4))) int32_t *Constant;
    return ((Constant)table)[min(key, last_key) >> a.seqs.page_shift];
  };

  // Where the lane's pieces of 16 keys lie, from the first key on: pages of 16
  // slots and more hold all of them in a row, and then one address does.  (Behind
  // the last key its own 16 are copied again.)
  const bool in_row = a.seqs.page_shift >= 4 && a.slot_stride < (1 << 24);
  uint32_t k_off[kCopies], v_off[kCopies];
#pragma unroll
  for (int j = 0; j < kCopies; ++j) {
    const int p = 64 * j + lane, key = p / CH, piece = p % CH;
    k_off[j] = (uint32_t)(key * (int)a.slot_stride * 2 + 16 * (piece ^ M::k_turn(key)));
    v_off[j] = (uint32_t)(key * (int)a.slot_stride * 2 + 16 * (piece ^ M::v_turn(key)));
  }
  const auto copy_tile = [&](int base, int slot) {
    if (base >= end) return;
    const uint32_t to = __builtin_amdgcn_readfirstlane(ring_at + slot * 2 * M::kBytes);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key0 = base + 16 * h;
      if (in_row) {
        const int64_t at = key_at(a, min(key0, last_key & ~15), page_at(key0)).at;
#pragma unroll
        for (int j = 0; j < kCopies; ++j) {
          copy_to_lds(ck + at, k_off[j], to + 1024 * (h * kCopies + j));
          copy_to_lds(cv + at, v_off[j], to + M::kBytes + 1024 * (h * kCopies + j));
        }
      } else {
#pragma unroll
        for (int j = 0; j < kCopies; ++j) {
          const int p = 64 * j + lane, key = p / CH, piece = p % CH;
          const int64_t at = key_at(a, min(key0 + key, last_key), page_of(key0 + key)).at;
          copy_to_lds(ck + at + 16 * (piece ^ M::k_turn(key)), to + 1024 * (h * kCopies + j));
          copy_to_lds(cv + at + 16 * (piece ^ M::v_turn(key)), to + M::kBytes + 1024 * (h * kCopies + j));
        }
      }
    }
  };
  // Keys of the tile that are there, a bit each.
  const auto there_of = [&](int base) -> uint32_t {
    if (in_row) {
      uint32_t there = ~bits_from(end - base);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if ((unsigned)page_at(base + 16 * h) >= (unsigned)a.n_pages) there &= ~(0xffffu << (16 * h));
      return __builtin_amdgcn_readfirstlane(there);
    }
    const int key = base + (lane & 31);
    return (uint32_t)__ballot((unsigned)page_of(key) < (unsigned)a.n_pages && key < end);
  };

  const int first = begin + 32 * wave;
#pragma unroll
  for (int i = 0; i < S; ++i) copy_tile(first + i * kStep, i);

  // the lane's q row
  const int row = it.tile * kFewRows + c, tok = row / a.group, q_head = head * a.group + row % a.group;
  const bool real = row < it.n * a.group;
  const int pos = it.len - it.n + tok;
  const int see_lo = first_seen(a, pos), see_hi = real ? end_seen(a, pos, it.len) : 0;
  V8 q[ST][NT];
  float scale = a.scale;
  int more = 0;
  {
    float x[ST][8];
    float most = 0.0f;
#pragma unroll
    for (int t = 0; t < ST; ++t) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[t][i] = 0.0f;
      if (real)
        load_as(a.q.type, a.q.p, (it.start + tok) * a.q.tok_stride + q_head * a.q.head_stride + 32 * t + 8 * g, x[t]);
#pragma unroll
      for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(x[t][i]));
    }
    if (T == QG_F16 && NT > 1) {
      const int e = row_exponent(max_of_row16(most)) - K::kRowTop;
      const RowScale by = row_scale(scale, e);
      scale = by.scale;
      more = by.more;
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[t][i] = ldexpf(x[t][i], -e);
    }
#pragma unroll
    for (int t = 0; t < ST; ++t) row_terms_of<T, NT>(x[t], q[t]);
  }

  const bool scaled_twice = T == QG_F16 && NT > 1 && __any(more > 0);
  f32x4 o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = f32x4{0, 0, 0, 0};
  float m = -kInf, l = 0.0f;
  bool odd_values = false;

  const auto all_see = [&](int base, uint32_t there) {
    return base >= range.all_lo && base + 32 <= range.all_hi && there == ~0u;
  };
  // Bit j: the lane's row sees key 4 g + j of those from base on, or 12 + 4 g + j from bit 4 on.
  const auto seen_of = [&](int base, uint32_t there) {
    const uint32_t in = (there & bits_from(see_lo - base) & ~bits_from(see_hi - base)) >> (4 * g);
    return (in & 15) | (in >> 12 & 0xf0);
  };
  const auto compute = [&](int base, uint8_t *tk) {
    uint8_t *const tv = tk + M::kBytes;
    f32x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const V8 key = *(const V8 *)(tk + (16 * u + c) * 2 * D + 16 * ((4 * t + g) ^ M::k_turn(c)));
#pragma unroll
        for (int k = 0; k < NT; ++k) s[u] = K::mfma16(key, q[t][k], s[u]);
      }
    float p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = s[j / 4][j & 3];
    if (scaled_twice) {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = ldexpf(p[j], more);
    }
    const uint32_t there = there_of(base);
    if (!all_see(base, there)) {
      const uint32_t seen = seen_of(base, there);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float score = p[j];
        p[j] = seen >> j & 1 ? score : -kInf;
      }
      // what is not there weighs nothing, and may hold anything
      bool odd = false;
#pragma unroll
      for (int j = 0; j < CH / 2; ++j) {
        u32x4 *const at = (u32x4 *)(tv + 16 * (64 * j + lane));
        u32x4 w = *at;
        if (!(there >> ((64 * j + lane) / CH) & 1)) w = u32x4{0, 0, 0, 0};
        odd = odd || !(finite2<T>(w[0]) && finite2<T>(w[1]) && finite2<T>(w[2]) && finite2<T>(w[3]));
        *at = u32x4{only_finite2<T>(w[0]), only_finite2<T>(w[1]), only_finite2<T>(w[2]), only_finite2<T>(w[3])};
      }
      odd_values = odd_values || __any(odd);
    }
    float top = p[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) top = fmaxf(top, p[j]);
    top = fmaxf(m, max_of_row16(top) * scale - K::kTop);
    if (__any(top > m)) {
      const float f = top > m ? exp2_of(m - top) : 1.0f;  // (of m = -inf, 0)
      l *= f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f;
      m = top;
    }
    const float off = m == -kInf ? 0.0f : m;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = exp2_of(fmaf(p[j], scale, -off));
      l += p[j];
    }
    V8 w[NT];
    terms_of<T, NT>(p, w);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      // value 16 e + c of keys 4 g + .. and 16 more
      const int key = 4 * g + (c >> 2), piece = 2 * e + ((c >> 1) & 1);
      const uint8_t *at = tv + key * 2 * D + 16 * (piece ^ M::v_turn(key)) + 8 * (c & 1);
      typedef __attribute__((address_space(3))) s16x4 *Lds;
      struct {
        s16x4 x[2];
      } col = {{__builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(s16x4 *)at),
                __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(s16x4 *)(at + 32 * D))}};
#pragma unroll
      for (int k = 0; k < NT; ++k) o[e] = K::mfma16(__builtin_bit_cast(V8, col), w[k], o[e]);
    }
  };

  int slot = 0;
  for (int base = first; base < end; base += kStep) {
    if (base + (S - 1) * kStep < end) wait_copies<(S - 1) * kTileCopies>();
    else wait_copies<0>();
    compute(base, ring + slot * 2 * M::kBytes);
    wait_reads();
    copy_tile(base + S * kStep, slot);
    slot = slot + 1 < S ? slot + 1 : 0;
  }
  if (odd_values) {
    for (int base = first; base < end; base += kStep) {
      const uint32_t there = there_of(base);
      if (all_see(base, there)) continue;
      const uint32_t seen = seen_of(base, there);
      int64_t at[8];
      u32x4 ones = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = min(base + 16 * (j / 4) + 4 * g + (j & 3), last_key);
        at[j] = key_at(a, key, page_of(key)).at;
        ones[j / 2] |= (seen >> j & 1 ? K::kOne : 0) << (16 * (j & 1));
      }
      for (int kind = kNan; kind <= kDown; ++kind) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          u32x4 is = {0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < 8; ++j)
            is[j / 2] |= is_kind<T>(*(const uint16_t *)(cv + at[j] + 2 * (16 * e + c)), kind) << (16 * (j & 1));
          const f32x4 n = K::mfma16(__builtin_bit_cast(V8, is), __builtin_bit_cast(V8, ones), f32x4{0, 0, 0, 0});
#pragma unroll
          for (int i = 0; i < 4; ++i) o[e][i] += of_kind(n[i], kind);
        }
      }
    }
  }

  // the waves' sums joined, 16 lanes a row
  l = sum_of_row16(l);
  if (g == 0) stats[wave][c] = make_float2(m, l);
  __syncthreads();
  float *const sums = (float *)lds;
#pragma unroll
  for (int e = 0; e < E; ++e) *(f32x4 *)(sums + (wave * kFewRows + c) * kStride + 16 * e + 4 * g) = o[e];
  __syncthreads();
#pragma unroll
  for (int r0 = 0; r0 < kFewRows; r0 += 4 * W) {
    const int r = r0 + (threadIdx.x >> 4), at = (threadIdx.x & 15) * E;
    const int out_row = it.tile * kFewRows + r;
    if (out_row >= it.n * a.group) return;
    float top = -kInf;
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, stats[w][r].x);
    float total = 0.0f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = stats[w][r].x == -kInf ? 0.0f : exp2_of(stats[w][r].x - top);
      total += stats[w][r].y * f;
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] += sums[(w * kFewRows + r) * kStride + at + e] * f;
    }
    if (it.parts == 1) {
      const int64_t t = it.start + out_row / a.group;
      const int h = head * a.group + out_row % a.group;
      float f, lse;
      bool none;
      finish_row(a, h, top, total, f, none, lse);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = none ? 0.0f : v[e] * f;
      store_row(a.out, t, h, at, v);
      if (a.lse && (threadIdx.x & 15) == 0) a.lse[t * a.group * a.kv_heads + h] = lse;
    } else {
      const int64_t pr = ((int64_t)(it.first + it.part) * a.kv_heads + head) * kFewRows + r;
#pragma unroll
      for (int e = 0; e < E; ++e) a.part[pr * D + at + e] = v[e];
      if ((threadIdx.x & 15) == 0) ((float2 *)(a.part + a.part_rows * D))[pr] = make_float2(top, total);
    }
  }
}

// ---------------------------------------------------------------------------
// Many rows: tiles of 128, 32 to a wave.  Bound by the matrix cores and by the
// softmax beside them.  Keys and values come in tiles of KT through LDS, the
// next tile's copies (HBM or L2 -> LDS, asynchronous, 16 bytes a lane) under way
// while one is computed.  32 x 32 x 16 instructions: a wave's q rows are their 32
// columns; K^T comes by 16-byte reads, V^T by the transposing 8-byte ones, whose
// four keys a lane are those of the scores' layout.
// Places of a row's pieces are exchanged as above.
// 8192 tokens, 32 heads over 8 of 128: 543 us, 1.01 PFLOP/s; its matrix
// instructions alone, without copies, reads of LDS and softmax, take 372.  The
// next scores computed beside a softmax (keys a tile further ahead), reads of
// LDS ordered ahead of the products, raised priorities: no gain.  A copy's
// addresses from one of its page, by the scalar unit, instead of one a lane:
// 704 to 608; the rows that see the most first: 608 to 565; 16 places exchanged
// for K, not 8: to 550.
// The running maximum follows only when a row's grows by more than 8 (in powers
// of 2): until then weights up to 256 times as large are as exact, and the sums
// need no factor.  (So those of fp16 are lost below 2^-32 of the largest, and a
// maximum's own weight in bf16 is 2^-8, as larger ones than 1 would make the sums
// of values near fp32's end infinite.)
// ---------------------------------------------------------------------------

constexpr int kManyWaves = 4, kManyRows = 32 * kManyWaves, kManyPiece = 64;
constexpr float kSlack = 8.0f;

template <int D> struct ManyTile {
  static constexpr int KT = D <= 128 ? 64 : 32;  // keys
  static constexpr int CH = D / 8;               // pieces of a row
  static constexpr int kBytes = KT * D * 2;
  static constexpr int kBanks = D / 2 % 64;      // where the next row begins
  static __host__ __device__ constexpr int k_turn(int key) {
    return kBanks == 0 ? key & 15 : kBanks == 32 ? (key >> 1) & 7 : (key >> 2) & 3;
  }
  static __host__ __device__ constexpr int v_turn(int key) {
    return kBanks == 0 ? (key & 3) << 2 : kBanks == 32 ? ((key >> 1) & 1) << 2 : 0;
  }
};

// The largest, the sum of a value and the one 32 lanes away.
__device__ __forceinline__ float max_of_row32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_of_row32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Waves a SIMD: as many as their sums and rows leave registers for.
constexpr int many_waves(int dim, int terms) { return dim <= 96 && terms == 1 ? 3 : dim * (1 + terms) <= 256 ? 2 : 1; }

template <int T, int D, int NT>
__global__ void __launch_bounds__(64 * kManyWaves, many_waves(D, NT)) attend_many_kernel(AttendArgs a, int64_t group0) {
  using K = Kind<T>;
  using V8 = typename K::V8;
  using M = ManyTile<D>;
  constexpr int KT = M::KT, CH = M::CH, U = KT / 32, ST = D / 16, DT = D / 32;
  constexpr float kAbove = K::kTop - kSlack;  // log2 of the running maximum's own weight
  // a wave copies a quarter of a tile's keys
  constexpr int kKeys = KT / kManyWaves, kCopies = (kKeys * CH + 63) / 64;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][2][M::kBytes];  // of a tile: K, V

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 31, h = lane >> 5;
  const int number = (int)((group0 + blockIdx.x) / a.kv_heads);
  const int head = (int)(group0 + blockIdx.x - (int64_t)number * a.kv_heads);
  const Item it = Plan<kManyRows, kManyPiece>(a).template find<false>(number);
  if (it.parts == 0) return;
  const Range range = range_of<kManyRows>(a, it);
  const int lo = range.lo & ~31, pieces = max(0, (int)(((int64_t)range.hi - lo + kManyPiece - 1) / kManyPiece));
  const int share = (pieces + it.parts - 1) / it.parts;
  const int begin = lo + min(pieces, it.part * share) * kManyPiece;
  const int end = min(range.hi, lo + min(pieces, (it.part + 1) * share) * kManyPiece);

  // the lane's q row, and what the wave's rows see
  const int row0 = it.tile * kManyRows + 32 * wave, rows = it.n * a.group;
  const int row = row0 + c, tok = row / a.group, q_head = head * a.group + row % a.group;
  const bool real = row < rows;
  const int old = it.len - it.n, pos = old + tok;
  const int see_lo = first_seen(a, pos), see_hi = real ? end_seen(a, pos, it.len) : 0;
  const int first_tok = row0 / a.group, last_tok = (min(row0 + 32, rows) - 1) / a.group;
  const int wave_lo = first_seen(a, old + first_tok);
  const int wave_hi = row0 < rows ? end_seen(a, old + last_tok, it.len) : 0;
  const int whole_lo = first_seen(a, old + last_tok), whole_hi = end_seen(a, old + first_tok, it.len);
  const uint8_t *ck = (const uint8_t *)(a.k + head * a.head_stride), *cv = (const uint8_t *)(a.v + head * a.head_stride);
  const int32_t *table = a.seqs.tables + it.s * a.seqs.max_pages;
  const int last_key = max(end - 1, 0);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)&lds[0][0][0];

  // Lane i holds the page of a tile's key i.
  const auto page_of = [&](int base) {
    return base < end ? table[min(base + (lane & (KT - 1)), last_key) >> a.seqs.page_shift] : -1;
  };
  // Keys of the tile that are there, a bit each.
  const auto there_of = [&](int base, int page) {
    return __ballot((unsigned)page < (unsigned)a.n_pages && base + (lane & (KT - 1)) < end);
  };
  // Where the lane's pieces of the wave's keys lie, from the first key on: pages
  // of kKeys slots and more hold all of them in a row, and then one address does.
  // (Behind the last key its own kKeys are copied again.)
  const bool in_row = a.seqs.page_shift >= log2_of(kKeys) && a.slot_stride < (1 << 24);
  uint32_t k_off[kCopies], v_off[kCopies];
#pragma unroll
  for (int j = 0; j < kCopies; ++j) {
    const int p = 64 * j + lane, key = min(p / CH, kKeys - 1), piece = p % CH;
    k_off[j] = (uint32_t)(key * (int)a.slot_stride * 2 + 16 * (piece ^ M::k_turn(kKeys * wave + key)));
    v_off[j] = (uint32_t)(key * (int)a.slot_stride * 2 + 16 * (piece ^ M::v_turn(kKeys * wave + key)));
  }
  const int first_key = __builtin_amdgcn_readfirstlane(kKeys * wave);
  const auto copy_tile = [&](int base, int page, int buf) {
    if (base >= end) return;
    const uint32_t to = __builtin_amdgcn_readfirstlane(lds0 + buf * 2 * M::kBytes + first_key * CH * 16);
    if (in_row) {
      const int64_t at =
          key_at(a, min(base + first_key, last_key & -kKeys), __builtin_amdgcn_readlane(page, first_key)).at;
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        if (kCopies * 64 > kKeys * CH && 64 * j + lane >= kKeys * CH) break;
        copy_to_lds(ck + at, k_off[j], to + 1024 * j);
        copy_to_lds(cv + at, v_off[j], to + M::kBytes + 1024 * j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        const int p = 64 * j + lane, key = min(p / CH, kKeys - 1) + first_key, piece = p % CH;
        const int64_t at = key_at(a, min(base + key, last_key), __shfl(page, key)).at;
        if (kCopies * 64 > kKeys * CH && p >= kKeys * CH) break;
        copy_to_lds(ck + at + 16 * (piece ^ M::k_turn(key)), to + 1024 * j);
        copy_to_lds(cv + at + 16 * (piece ^ M::v_turn(key)), to + M::kBytes + 1024 * j);
      }
    }
  };

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = -kInf, l = 0.0f;

  constexpr uint64_t kAll = KT == 64 ? ~0ull : (1ull << KT) - 1;
  const auto all_see = [&](int base, uint64_t now) {
    return base >= range.all_lo && base + KT <= range.all_hi && (now & kAll) == kAll;
  };
  // Bit 8 (i / 4) + i % 4: the lane's row sees key i of its own of the 32 from base + 32 u on.
  const auto seen = [&](int base, uint64_t now, int u) {
    return ((uint32_t)(now >> (32 * u)) & bits_from(see_lo - base - 32 * u) & ~bits_from(see_hi - base - 32 * u)) >>
           (4 * h);
  };
  bool odd_values = false;
  int page = page_of(begin);
  uint64_t there = there_of(begin, page);
  copy_tile(begin, page, 0);
  page = page_of(begin + KT);

  V8 q[ST][NT];
  float scale = a.scale;
  int more = 0;
  {
    float x[ST][8];
    float most = 0.0f;
#pragma unroll
    for (int t = 0; t < ST; ++t) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[t][i] = 0.0f;
      if (real)
        load_as(a.q.type, a.q.p, (it.start + tok) * a.q.tok_stride + q_head * a.q.head_stride + 16 * t + 8 * h, x[t]);
#pragma unroll
      for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(x[t][i]));
    }
    if (T == QG_F16 && NT > 1) {
      const int e = row_exponent(max_of_row32(most)) - K::kRowTop;
      const RowScale by = row_scale(scale, e);
      scale = by.scale;
      more = by.more;
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[t][i] = ldexpf(x[t][i], -e);
    }
#pragma unroll
    for (int t = 0; t < ST; ++t) row_terms_of<T, NT>(x[t], q[t]);
  }
  const bool scaled_twice = T == QG_F16 && NT > 1 && __any(more > 0);
  int buf = 0;
  for (int base = begin; base < end; base += KT, buf ^= 1) {
    wait_copies<0>();
    __syncthreads();
    uint8_t *tk = lds[buf][0], *tv = lds[buf][1];
    const uint64_t now = there;
    if (!all_see(base, now)) {
      bool odd = false;
      // what is not there weighs nothing, and may hold anything
      for (int i = threadIdx.x; i < KT * CH; i += 64 * kManyWaves) {
        u32x4 *const at = (u32x4 *)(tv + 16 * i);
        if (!(now >> (i / CH) & 1)) *at = u32x4{0, 0, 0, 0};
        const u32x4 w = *at;
        odd = odd || !(finite2<T>(w[0]) && finite2<T>(w[1]) && finite2<T>(w[2]) && finite2<T>(w[3]));
      }
      odd = __syncthreads_or(odd);
      if (odd) {
        odd_values = true;
        for (int i = threadIdx.x; i < KT * CH; i += 64 * kManyWaves) {
          u32x4 *const at = (u32x4 *)(tv + 16 * i);
          const u32x4 w = *at;
          *at = u32x4{only_finite2<T>(w[0]), only_finite2<T>(w[1]), only_finite2<T>(w[2]), only_finite2<T>(w[3])};
        }
        __syncthreads();
      }
    }
    there = there_of(base + KT, page);
    copy_tile(base + KT, page, buf ^ 1);
    page = page_of(base + 2 * KT);
    if (base >= wave_hi || base + KT <= wave_lo) continue;

    f32x16 s[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const V8 key = *(const V8 *)(tk + (32 * u + c) * 2 * D + 16 * ((2 * t + h) ^ M::k_turn(c)));
#pragma unroll
        for (int k = 0; k < NT; ++k) s[u] = K::mfma32(key, q[t][k], s[u]);
      }
    if (scaled_twice) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[u][i] = ldexpf(s[u][i], more);
    }
    const bool whole = base >= whole_lo && base + KT <= whole_hi && (now & kAll) == kAll;
    if (!whole) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t mine = seen(base, now, u);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float x = s[u][i];
          s[u][i] = mine & 1u << (8 * (i / 4) + (i & 3)) ? x : -kInf;
        }
      }
    }
    float top = s[0][0];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
    top = max_of_row32(top) * scale - kAbove;
    if (__any(top > m + kSlack)) {
      const float f = top > m ? exp2_of(m - top) : 1.0f;  // (of m = -inf, 0)
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= f;
      m = fmaxf(m, top);
    }
    const float off = m == -kInf ? 0.0f : m;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[u][i] = exp2_of(fmaf(s[u][i], scale, -off));
        sum += s[u][i];
      }
      l += sum;
    }
#pragma unroll
    for (int t = 0; t < KT / 16; ++t) {
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = s[t / 2][8 * (t & 1) + i];
      V8 w[NT];
      terms_of<T, NT>(p, w);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        // values 32 d + c of keys 16 t + 4 h + .. and 8 more
        const int a16 = lane & 15, key = 16 * t + 4 * h + (a16 >> 2);
        const int piece = 4 * d + 2 * ((lane >> 4) & 1) + ((a16 >> 1) & 1);
        const uint8_t *at = tv + key * 2 * D + 16 * (piece ^ M::v_turn(a16 >> 2)) + 8 * (a16 & 1);
        typedef __attribute__((address_space(3))) s16x4 *Lds;
        struct {
          s16x4 x[2];
        } col = {{__builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(s16x4 *)at),
                  __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(s16x4 *)(at + 16 * D))}};
#pragma unroll
        for (int k = 0; k < NT; ++k) o[d] = K::mfma32(__builtin_bit_cast(V8, col), w[k], o[d]);
      }
    }
  }

  if (odd_values) {
    for (int base = begin; base < end; base += KT) {
      const uint64_t now = there_of(base, page_of(base));
      if (all_see(base, now) || base >= wave_hi || base + KT <= wave_lo) continue;
      for (int kind = kNan; kind <= kDown; ++kind) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          f32x16 n;
#pragma unroll
          for (int i = 0; i < 16; ++i) n[i] = 0.0f;
          for (int t = 0; t < KT / 16; ++t) {
            u32x4 is = {0, 0, 0, 0}, ones = {0, 0, 0, 0};
            const uint32_t mine = seen(base, now, t / 2) >> (16 * (t & 1));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int key = min(base + 16 * t + 8 * (j / 4) + 4 * h + (j & 3), last_key);
              const uint32_t v = *(const uint16_t *)(
                  cv + key_at(a, key, table[key >> a.seqs.page_shift]).at + 2 * (32 * d + c));
              is[j / 2] |= is_kind<T>(v, kind) << (16 * (j & 1));
              ones[j / 2] |= (mine & 1u << (8 * (j / 4) + (j & 3)) ? K::kOne : 0) << (16 * (j & 1));
            }
            n = K::mfma32(__builtin_bit_cast(V8, is), __builtin_bit_cast(V8, ones), n);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][i] += of_kind(n[i], kind);
        }
      }
    }
  }

  l = sum_of_row32(l);
  if (!real) return;
  if (it.parts == 1) {
    const int64_t t = it.start + tok;
    float f, lse;
    bool none;
    finish_row(a, q_head, m, l, f, none, lse);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = none ? 0.0f : o[d][4 * i + j] * f;
        store_row(a.out, t, q_head, 32 * d + 8 * i + 4 * h, v);
      }
    if (a.lse && h == 0) a.lse[t * a.group * a.kv_heads + q_head] = lse;
  } else {
    const int64_t pr = ((int64_t)(it.first + it.part) * a.kv_heads + head) * kManyRows + 32 * wave + c;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *(f32x4 *)(a.part + pr * D + 32 * d + 8 * i + 4 * h) =
            f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
    if (h == 0) ((float2 *)(a.part + a.part_rows * D))[pr] = make_float2(m, l);
  }
}

// ---------------------------------------------------------------------------
// The parts of a tile joined, where there are several.  A workgroup takes
// `rows` of the tile's rows (all 16 of few, or one where there are few tiles and
// so may be hundreds of parts; all 128 of many, or 16 where there are few tiles):
// groups of its lanes take a row's every so many parts, 4 values a lane.
// ---------------------------------------------------------------------------

template <int D, int ROWS, int PIECE>
__global__ void __launch_bounds__(256) attend_join_kernel(AttendArgs a, int rows, int64_t group0) {
  constexpr int kLanes = D / 4 <= 8 ? 8 : D / 4 <= 16 ? 16 : D / 4 <= 32 ? 32 : 64, kGroups = 256 / kLanes;
  __shared__ f32x4 sums[kGroups][kLanes];
  __shared__ float2 stats_of[kGroups];
  const int64_t group = group0 + blockIdx.x;
  const int per = ROWS / rows;  // workgroups of a tile
  const int sub = (int)(group / a.kv_heads), head = (int)(group - (int64_t)sub * a.kv_heads);
  const Item it = Plan<ROWS, PIECE>(a).template find<true>(sub / per);
  if (it.parts < 2) return;
  // (starts that do not rise give more rows than the workspace is for)
  if (it.first < 0 || ((int64_t)it.first + it.parts) * a.kv_heads * ROWS > a.part_rows) return;
  const int row0 = it.tile * ROWS + sub % per * rows, real = min(rows, it.n * a.group - row0);
  if (real <= 0) return;
  int each = kGroups;  // groups of a row
  while (each > 1 && (each * real > kGroups || each >= 2 * it.parts)) each /= 2;
  const int i = threadIdx.x / kLanes, at = 4 * (threadIdx.x % kLanes);
  const float2 *stats = (const float2 *)(a.part + a.part_rows * D);
  const int64_t step = (int64_t)a.kv_heads * ROWS;
  for (int r0 = 0; r0 < real; r0 += kGroups / each) {
    const int r = r0 + i / each, j = i % each, row = row0 + r;
    const int64_t first = ((int64_t)it.first * a.kv_heads + head) * ROWS + row - it.tile * ROWS;
    float m = -kInf, l = 0.0f;
    f32x4 v = {0, 0, 0, 0};
    if (r < real) {
      for (int p = j; p < it.parts; p += each) m = fmaxf(m, stats[first + p * step].x);
#pragma unroll 4
      for (int p = j; p < it.parts; p += each) {
        const float2 s = stats[first + p * step];
        const float f = s.x == -kInf ? 0.0f : exp2_of(s.x - m);
        l += s.y * f;
        if (at < D) v += *(const f32x4 *)(a.part + (first + p * step) * D + at) * f;
      }
    }
    if (each > 1) {
      sums[i][at / 4] = v;
      if (at == 0) stats_of[i] = make_float2(m, l);
      __syncthreads();
      if (j == 0) {
        float top = m;
        for (int k = 1; k < each; ++k) top = fmaxf(top, stats_of[i + k].x);
        const float f = m == -kInf ? 0.0f : exp2_of(m - top);
        l *= f;
        v *= f;
        for (int k = 1; k < each; ++k) {
          const float2 s = stats_of[i + k];
          const float fk = s.x == -kInf ? 0.0f : exp2_of(s.x - top);
          l += s.y * fk;
          v += sums[i + k][at / 4] * fk;
        }
        m = top;
      }
      __syncthreads();
    }
    if (r >= real || j > 0 || at >= D) continue;
    const int64_t t = it.start + row / a.group;
    const int h = head * a.group + row % a.group;
    float f, lse;
    bool none;
    finish_row(a, h, m, l, f, none, lse);
    float out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = none ? 0.0f : v[i] * f;
    store_row(a.out, t, h, at, out);
    if (a.lse && at == 0) a.lse[t * a.group * a.kv_heads + h] = lse;
  }
}

// A call's shape: the rows of a tile, the most tiles and parts its sequences can have.
struct AttendShape {
  int64_t tiles, parts;
  int rows, target;
};

template <int T> hipError_t launch_attend(const AttendArgs &a, const AttendShape &s, int dim, bool wide,
                                          hipStream_t stream);

}  // namespace qgemv_kv
