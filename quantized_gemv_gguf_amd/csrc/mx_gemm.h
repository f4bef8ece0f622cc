// mx_gemm.h -- products of many tokens with MXFP4 weights on gfx950's matrix
// cores: y[t][n] = sum_k x[t][k] W[n][k], dense or for tokens sorted by expert,
// single or as a SwiGLU pair.  One translation unit per activation type
// (mx_f32, mx_f16, mx_bf16, mx_fp4).
//
// Operands.  W is operand A (rows n), x operand B (columns t), so a lane's
// four sums are four consecutive n of one token.  An MXFP4 block is 16 bytes
// of codes and one scale byte per 32 weights, and a lane of the K = 128 scaled
// instruction holds exactly one block: lane (i, g) = row i, block g of the
// step.  The order of k inside a block is free as long as both sides share it,
// so GGUF's split-half nibbles are used as they lie:
//   MXFP4 x   v_mfma_scale_f32_16x16x128_f8f6f4 on the blocks of both sides.
//   float x   four v_mfma_f32_16x16x32_bf16 per step: the j-th takes word j of
//             each lane's block, i.e. elements (4j + b, 16 + 4j + b), b < 4, as
//             pairs out of v_cvt_scalef32_pk_bf16_fp4 (exact: an E2M1 value
//             times a power of two), and x is laid into LDS in that order.
//             fp32 x is the exact sum of three bf16 terms (8 bits each,
//             truncated, so no term rounds), fp16 of two, bf16 of one: every
//             product is exact and only the fp32 sums round.  (Bits of fp32 x
//             below 2^-133, the least bf16 subnormal, are cut off.)  Weights of
//             2^128 and more, which bf16 does not hold: see huge_block.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "qgemv_mx.h"

namespace qgemv_mx {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct MxArgs {
  const uint8_t *w, *w2;   // first row of the window (experts: of the stack); the up matrix of a pair
  const uint8_t *x;
  void *y;
  const int32_t *offsets;  // experts: n_expert + 1; null: one dense product
  const int32_t *slots;    // null: row p of x
  int64_t expert_bytes;    // bytes from one expert's matrix to the next
  int64_t x_bytes;         // bytes from one row of x to the next
  int64_t y_stride;        // elements
  int32_t row_bytes;       // 17 nb
  int32_t nb;              // blocks per row
  int32_t n;               // output rows of a matrix
  int32_t places;          // rows of y
  int32_t x_rows;
  int32_t n_expert, n_sel;
  int32_t y_type;
  int32_t tiles_n, tiles;  // tiles along n; all tiles of the grid (an upper bound for experts)
};

// Activation kinds: bf16 terms per value, 0 for MXFP4.
enum { kFp4 = 0, kBf16 = 1, kF16 = 2, kF32 = 3 };

// Tile of one workgroup, in order of tokens: which expert, first place, places.
struct Tile {
  int expert, n0, m0, m_end;
};

// This workgroup's tile.  Workgroups go to the eight XCDs in turn; each XCD
// takes one contiguous run of the tiles there are (of experts: fewer than the
// grid's bound, so the runs are cut by the count found here), so that
// neighbours in the order below share an L2.  Order: experts; within an expert
// bands of eight token tiles; within a band tile rows n, and innermost the
// band's token tiles, so one weight tile is read by up to eight neighbours and
// the band's tokens stay in the XCD's L2 for the whole sweep over n.
// Every wave finds its tile by itself: lane l sums the token tiles of its run
// of experts, a scan over the lanes gives the first tile of each run, and the
// lane whose run holds the tile walks it.
template <int TM>
__device__ __forceinline__ bool find_tile(const MxArgs &a, int tn_rows, Tile *t) {
  const int lane = threadIdx.x & 63;
  const int run = (a.n_expert + 63) >> 6;
  const int e0 = min(lane * run, a.n_expert), e1 = min(e0 + run, a.n_expert);
  auto at = [&](int i) { return min(max(a.offsets[i], 0), a.places); };
  int mine = 0, upto = 0, tiles = a.tiles;
  if (a.offsets) {
    int o = e0 < e1 ? at(e0) : 0;
#pragma unroll 4
    for (int i = e0; i < e1; ++i) {
      const int q = at(i + 1);
      mine += (max(q - o, 0) + TM - 1) / TM;
      o = q;
    }
    upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    tiles = min(tiles, __builtin_amdgcn_readlane(upto, 63) * a.tiles_n);
  }
  const int per = (tiles + 7) >> 3, at_xcd = (int)(blockIdx.x >> 3);
  const int id = (int)(blockIdx.x & 7) * per + at_xcd;
  if (at_xcd >= per || id >= tiles) return false;
  int e = 0, lo = 0, hi = a.places, rem = id;
  if (a.offsets) {
    const int mt = id / a.tiles_n;  // token tiles before this one, over all experts
    const uint64_t past = __ballot(upto > mt);
    if (!past) return false;
    const int src = __builtin_ctzll(past);
    int first = __builtin_amdgcn_readlane(upto - mine, src);
    e = __builtin_amdgcn_readlane(e0, src);
    const int last = __builtin_amdgcn_readlane(e1, src);
    lo = at(e);
    hi = at(e + 1);
    for (;;) {
      const int here = (max(hi - lo, 0) + TM - 1) / TM;
      if (mt < first + here || e + 1 >= last) break;
      first += here;
      ++e;
      lo = hi;
      hi = at(e + 1);
    }
    e = __builtin_amdgcn_readfirstlane(e);
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    rem = id - __builtin_amdgcn_readfirstlane(first) * a.tiles_n;
  }
  const int mtiles = (hi - lo + TM - 1) / TM;
  const int band = rem / (8 * a.tiles_n);
  const int width = min(8, mtiles - 8 * band);
  if (width <= 0) return false;
  const int r = rem - band * 8 * a.tiles_n;
  const int tn = r / width, tm = 8 * band + r % width;
  if (tn >= a.tiles_n) return false;
  t->expert = e;
  t->n0 = tn * tn_rows;
  t->m0 = lo + tm * TM;
  t->m_end = min(hi, t->m0 + TM);
  return true;
}

// silu(g) u with the hardware exp2 and reciprocal, as qgemv_silu_mul.
__device__ __forceinline__ float silu_times(float g, float u) {
  const float e = __builtin_amdgcn_exp2f(-g * 1.44269504088896341f);
  return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // round to nearest even
  bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  h2 v = {(_Float16)a, (_Float16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// Four consecutive n of one token, `left` of them inside the matrix.
__device__ __forceinline__ void store4(const MxArgs &a, int place, int n, int left, f32x4 v) {
  const int64_t at = (int64_t)place * a.y_stride + n;
  if (a.y_type == QG_F32) {
    float *p = (float *)a.y + at;
    if (left >= 4) __builtin_memcpy(p, &v, 16);
    else
#pragma unroll
      for (int r = 0; r < 3; ++r)
        if (r < left) p[r] = v[r];
  } else {
    uint16_t *p = (uint16_t *)a.y + at;
    const bool h = a.y_type == QG_F16;
    const u32x2 b = {h ? pack_f16(v.x, v.y) : pack_bf16(v.x, v.y), h ? pack_f16(v.z, v.w) : pack_bf16(v.z, v.w)};
    if (left >= 4) __builtin_memcpy(p, &b, 8);
    else
#pragma unroll
      for (int r = 0; r < 3; ++r)
        if (r < left) p[r] = (uint16_t)(b[r >> 1] >> (16 * (r & 1)));
  }
}

// A workgroup's outputs through LDS, a row of fragments (16 tokens of each of
// the WM waves) at a time, so that a store instruction writes whole lines of
// y: a lane's own eight bytes would leave each line to eight instructions.
// (4096 x 24576 bf16 outputs of MXFP4 tokens, k = 6144: 480 us with the lanes'
// own stores, 411 so; below 64 tokens a workgroup, 128 of float tokens, the
// lanes' own stores are no slower and leave more registers.)  ES: bytes of an
// output.
template <typename S, int ES, typename V, typename A>
__device__ __forceinline__ void store_rows(const MxArgs &a, const Tile &tile, uint8_t *lds, int wn, int wm, int i, int g,
                                           V outputs, A absent) {
  constexpr int kPitch = S::TN * ES + 16, kLanes = S::TN * ES / 16;  // 16-byte pieces of a token's row
  constexpr int kTokens = 16 * S::kWM;
  const int left = a.n - tile.n0;
#pragma unroll
  for (int m = 0; m < S::kFM; ++m) {
    __syncthreads();
#pragma unroll
    for (int n = 0; n < S::kFN; ++n) {
      const f32x4 v = outputs(n, m);
      uint8_t *at = lds + (16 * wm + i) * kPitch + (16 * (wn * S::kFN + n) + 4 * g) * ES;
      if constexpr (ES == 4) {
        *(f32x4 *)at = v;
      } else {
        const bool h = a.y_type == QG_F16;
        *(u32x2 *)at = u32x2{h ? pack_f16(v.x, v.y) : pack_bf16(v.x, v.y), h ? pack_f16(v.z, v.w) : pack_bf16(v.z, v.w)};
      }
    }
    __syncthreads();
    for (int q = threadIdx.x; q < kTokens * kLanes; q += S::kThreads) {
      const int tok = q / kLanes, piece = q % kLanes, col = piece * (16 / ES);
      const int p = tile.m0 + 16 * ((tok >> 4) * S::kFM + m) + (tok & 15);
      if (p >= tile.m_end || col >= left) continue;
      u32x4 v = *(const u32x4 *)(lds + tok * kPitch + 16 * piece);
      if (absent(p)) v = u32x4{0, 0, 0, 0};
      uint8_t *y = (uint8_t *)a.y + ((int64_t)p * a.y_stride + tile.n0 + col) * ES;
      if (col + 16 / ES <= left) __builtin_memcpy(y, &v, 16);
      else
#pragma unroll
        for (int k = 0; k < 16 / ES - 1; ++k)
          if (col + k < left) {
            if constexpr (ES == 4) ((uint32_t *)y)[k] = v[k];
            else ((uint16_t *)y)[k] = (uint16_t)(v[k >> 1] >> (16 * (k & 1)));
          }
    }
  }
}

// The bf16 terms of eight values in the lane order of the codes' word: element
// pairs (lo[b], hi[b]), lo = four values from 4q, hi = four from 16 + 4q.
// Terms are cut, not rounded: the rest is exact.
// What a lane loads of a block: fp32 its own four and four values, two 16-byte
// loads; bf16 and fp16 values 8q .. 8q + 7 in one, of which lanes q and q ^ 2
// exchange halves, so that lane q holds word 2 (q & 1) + (q >> 1).
template <int XK> struct XRaw;
template <> struct XRaw<kBf16> { u32x2 a, b; };
template <> struct XRaw<kF16> { u32x2 a, b; };
template <> struct XRaw<kF32> { f32x4 lo, hi; };

template <int XK> __device__ __forceinline__ int x_word(int q) { return XK == kF32 ? q : 2 * (q & 1) + (q >> 1); }

__device__ __forceinline__ uint32_t from_lane_xor2(uint32_t v) {  // lanes of a quad: 2, 3, 0, 1
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true);
}

template <int XK>
__device__ __forceinline__ void x_load(const uint8_t *p, XRaw<XK> &r) {  // p: the block's values, q: lane % 4
  const int q = threadIdx.x & 3;
  if constexpr (XK == kF32) {
    __builtin_memcpy(&r.lo, p + 16 * q, 16);
    __builtin_memcpy(&r.hi, p + 16 * q + 64, 16);
  } else {
    u32x4 v;
    __builtin_memcpy(&v, p + 16 * q, 16);
    r.a = v.xy;
    r.b = v.zw;
  }
}

__device__ __forceinline__ uint32_t top_halves(uint32_t lo, uint32_t hi) {  // (lo >> 16) | (hi & 0xffff0000)
  return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

// v cut to its first bf16; *rest = v minus it, exactly: 0 for an infinity, and
// NaN for a NaN, which then stays one whatever the cut leaves of its payload.
__device__ __forceinline__ uint32_t cut(float v, float *rest, bool first) {
  const uint32_t h = __float_as_uint(v) & 0xffff0000u;
  *rest = v - __uint_as_float(h);
  if (first && __builtin_isinf(v)) *rest = 0.0f;
  return h;
}

template <int XK>
__device__ __forceinline__ void x_terms(const XRaw<XK> &r, u32x4 (&out)[XK]) {
  u32x2 l2, h2;
  if constexpr (XK != kF32) {
    const bool first = !(threadIdx.x & 2);
    const u32x2 give = first ? r.b : r.a;
    const u32x2 got = {from_lane_xor2(give.x), from_lane_xor2(give.y)};
    l2 = first ? r.a : got;
    h2 = first ? got : r.b;
  }
  if constexpr (XK == kBf16) {
    out[0] = u32x4{__builtin_amdgcn_perm(h2.x, l2.x, 0x05040100u), __builtin_amdgcn_perm(h2.x, l2.x, 0x07060302u),
                   __builtin_amdgcn_perm(h2.y, l2.y, 0x05040100u), __builtin_amdgcn_perm(h2.y, l2.y, 0x07060302u)};
  } else {
    float lo[4], hi[4];
    if constexpr (XK == kF16) {
      typedef _Float16 h4 __attribute__((ext_vector_type(4)));
      const h4 l = __builtin_bit_cast(h4, l2), h = __builtin_bit_cast(h4, h2);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        lo[b] = (float)l[b];
        hi[b] = (float)h[b];
      }
    } else {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        lo[b] = r.lo[b];
        hi[b] = r.hi[b];
      }
    }
#pragma unroll
    for (int t = 0; t < XK; ++t)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (t == XK - 1) {
          out[t][b] = top_halves(__float_as_uint(lo[b]), __float_as_uint(hi[b]));
        } else {
          float rl, rh;
          const uint32_t l = cut(lo[b], &rl, t == 0), h = cut(hi[b], &rh, t == 0);
          out[t][b] = top_halves(l, h);
          lo[b] = rl;
          hi[b] = rh;
        }
      }
  }
}

// A block at any address: 17-byte blocks start at any byte, and the five
// aligned words that hold one are read as words 0 .. 3 and 3 .. 4.  For a wave
// of 16 rows of four blocks, a compute unit's address unit takes 17 cycles for
// a 16-byte load on a word's boundary, 65 for one off it, 20 for the 8-byte
// load, and 37 for a load of the fifth word alone (which takes a cycle per
// line, not per four lanes).  The words lie inside the 16-byte granules that the block
// touches.
struct BlockRaw {
  u32x4 a;
  u32x2 c;
};
__device__ __forceinline__ void block_load(const uint8_t *words, BlockRaw &r) {
  const uint8_t *p = (const uint8_t *)__builtin_assume_aligned(words, 4);
  __builtin_memcpy(&r.a, p, 16);
  __builtin_memcpy(&r.c, p + 12, 8);
}
// The codes (bytes 1 .. 16) of a block that starts at byte `phase` (0 .. 3) of its words.
__device__ __forceinline__ u32x4 block_codes(const BlockRaw &r, uint32_t phase) {
  asm volatile("" : : "v"(r.c));  // (keeps the second load whole: only its last word is new)
  const uint32_t sel = 0x04030201u + 0x01010101u * phase;
  return u32x4{__builtin_amdgcn_perm(r.a.y, r.a.x, sel), __builtin_amdgcn_perm(r.a.z, r.a.y, sel),
               __builtin_amdgcn_perm(r.a.w, r.a.z, sel), __builtin_amdgcn_perm(r.c.y, r.a.w, sel)};
}
__device__ __forceinline__ uint32_t block_scale(const BlockRaw &r, uint32_t phase) { return r.a.x >> (8 * phase); }

// Word j of a lane's block as four bf16 pairs, scale included.
__device__ __forceinline__ bf16x8 weights8(uint32_t codes, float scale) {
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  const u32x4 v = {__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1),
                   __builtin_bit_cast(uint32_t, p2), __builtin_bit_cast(uint32_t, p3)};
  return __builtin_bit_cast(bf16x8, v);
}

// Byte f of packed scale bytes as the fp32 2^(e - 127) bit pattern the
// conversion takes its exponent from.
__device__ __forceinline__ float scale_of(uint32_t bytes, int f) {
  return __uint_as_float(((bytes >> (8 * f)) & 0xffu) << 23);
}

// Whether a block holds a value of 2^128 or more (codes 2, 3, 4 and 6 at scale
// 254, 4 and 6 at 253), an infinity in bf16.
__device__ __forceinline__ bool huge_block(const uint8_t *block) {
  const int e = block[0];
  if (e != 253 && e != 254) return false;
  uint32_t any = 0;  // third bit of each code: that, or that and the second
  for (int j = 1; j < 17; ++j) any |= e == 254 ? block[j] : block[j] & (block[j] << 1);
  return any & 0x44u;
}

// One output from the values in memory, in 64 bits: nb blocks against a row of x.
template <int XK>
__device__ __forceinline__ float one_output(const uint8_t *w, const uint8_t *x, int nb) {
  typedef std::conditional_t<XK == kF32, float, std::conditional_t<XK == kF16, _Float16, __bf16>> X;
  typedef float f2 __attribute__((ext_vector_type(2)));
  double sum = 0.0;
#pragma unroll 1
  for (int b = 0; b < nb; ++b, w += 17, x += 32 * sizeof(X)) {
    const uint64_t e = w[0];
    const double scale = __builtin_bit_cast(double, (e == 255 ? 0x7ffull : e + 896) << 52 | (e == 255));
#pragma unroll 4
    for (int j = 0; j < 16; ++j) {
      const f2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[1 + j], 1.0f, 0);  // low nibble, high nibble
      sum = fma((double)((const X *)x)[j], v.x * scale, sum);
      sum = fma((double)((const X *)x)[16 + j], v.y * scale, sum);
    }
  }
  return (float)sum;
}

// f(integral_constant<0>) ... f(integral_constant<N - 1>)
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>());
    each<N, I + 1>(f);
  }
}

// The tiled product.  A workgroup of WN x WM x WK waves owns 16 FN WN rows of W
// (of each of a pair) and 16 FM WM tokens; a wave 16 FN x 16 FM of them, over
// every WK-th group of four blocks (128 values), and the WK partial sums are
// added in order through LDS at the end.  A stage is KS such groups: the next
// stage's blocks and activations are loaded into registers while the current
// one, in LDS, is multiplied.  NBUF = 2: two stages in LDS, one barrier each.
// COLS: the bf16 terms of a few tokens lie in matrix columns of their own (five
// fp32 tokens, or eight fp16, in 16 columns) and are added at the end: a single
// token costs one matrix instruction, not one per term.
// LDS: codes [group][row][block], 16 bytes each, so a wave's fragment of 16
// rows is 1 KB read without conflicts; scale bytes of four fragments of 16
// rows in one word; groups of both padded so that what a wave writes at a time
// falls into different banks (23 bf16 tokens, 4096 rows of 11008: 14.7 us with
// the scales' groups in the same ones, 14.2 so); float x as [term][group][fragment][word j][token][block],
// the planes of words 64 bytes apart beyond their 1 KB so that a token's
// sixteen pieces are written to sixteen bank groups.
//
// What bounds it.  MXFP4 tokens, 4096 x 24576 outputs of k = 6144: 385 to 425 us,
// 2.9 to 3.2 PFLOP/s (a bf16 library product of 8192^3 runs at 1.1).  LDS is busy
// for 61% of that, the matrix cores for 36%, and 5.2 GB pass from L2 to the compute
// units, 13 TB/s: a stage's 136 bytes of a row are two lines of 128, of which
// the next stage fetches one again (stages of 128 values: 7.2 GB).  bf16 tokens,
// 2048 x 8192 outputs of k = 4096: 123 to 137 us, 1.0 to 1.1 PFLOP/s, a library
// product's rate.  fp32 tokens take three times the matrix instructions, 270 to
// 300 us.  4096 MXFP4 tokens x 4 of 128 experts, pair of 2880 x 2880: 530
// us, LDS 42% busy and 4.9 GB from L2; a sixth of it is the weights' way from
// memory (470 us instead of 570, in another shape, with one expert's weights for
// all).  Few tokens: the blocks' latency and, for fp32, the terms, which every
// workgroup makes anew.
template <int XK, bool PAIR, int FN, int FM, int WN, int WM, int WK, int KS, int NBUF, bool COLS = false>
struct MxTile {
  static constexpr int kThreads = 64 * WN * WM * WK;
  static constexpr int TN = 16 * FN * WN;
  static constexpr int kTerms = XK == kFp4 || COLS ? 1 : XK;   // of x in one matrix column
  static constexpr int kCols = COLS ? XK : 1;                  // matrix columns of one token
  static constexpr int TM = 16 * FM * WM / kCols;              // tokens
  static constexpr int kMats = PAIR ? 2 : 1;
  static constexpr int kWRows = TN * kMats;
  static constexpr int kBlk = 4 * KS;                          // blocks of a row per stage
  static constexpr int kRowStep = kThreads / kBlk;             // rows of W (of MXFP4 x) loaded at a time
  static constexpr int NW = kWRows / kRowStep;
  static constexpr int kTokStep = XK == kFp4 ? kRowStep : kRowStep / 4;
  static constexpr int NX = (TM + kTokStep - 1) / kTokStep;
  static constexpr int kWGroup = kWRows * 64 + 256 / KS;       // codes of one group, padded
  static constexpr int kWSPad = KS > 1 ? 256 / KS : 0;
  static constexpr int kWSGroup = (kWRows + 63) / 64 * 256 + kWSPad;  // its scales
  static constexpr int kPlane = 1024 + 64;                     // one word of 16 tokens, padded
  static constexpr int kXFrag = 4 * kPlane;
  static constexpr int kXGroup = XK == kFp4 ? TM * 64 + 256 / KS : FM * WM * kXFrag;
  static constexpr int kXSGroup = XK == kFp4 ? (TM + 63) / 64 * 256 + kWSPad : 0;
  static constexpr int kOffWS = KS * kWGroup, kOffX = kOffWS + KS * kWSGroup, kOffXS = kOffX + kTerms * KS * kXGroup;
  static constexpr int kStage = kOffXS + KS * kXSGroup;
  static constexpr int kRed = (WK - 1) * WN * WM * kMats * FN * FM * 1024;
  // larger tiles store their outputs by rows (store_rows)
  static constexpr bool kRows = WK == 1 && FM * WM > (XK == kFp4 ? 2 : 4);
  static constexpr int kFN = FN, kFM = FM, kWM = WM;
  // MXFP4 x, 128 registers of sums a lane: one loop for every stage (see there)
  static constexpr bool kOneLoop = XK == kFp4 && NBUF == 2 && kMats * FN * FM >= 32;
  static constexpr int kOut = kRows ? 16 * WM * (4 * TN + 16) : 0;
  static constexpr int kMost = kRed > kOut ? kRed : kOut;
  static constexpr int kLds = NBUF * kStage > kMost ? NBUF * kStage : kMost;
  static_assert(kThreads % kBlk == 0 && kWRows % kRowStep == 0, "a stage's blocks divide over the threads");
  static_assert(kRowStep % 4 == 0, "so do its activations, and a thread's rows share their alignment");
  static_assert(!PAIR || TN % kRowStep == 0, "a load's rows are of one matrix");
  static_assert(KS % WK == 0 && kLds <= 160 * 1024, "");
  static_assert(!COLS || (XK >= kF16 && FM == 1 && WM == 1), "columns of one fragment");
};

// Waves to a SIMD that the compiler has to leave registers for (0: its own
// choice).  bf16 tokens in eight waves: three workgroups to a compute unit, by
// itself it takes two registers more and leaves two.
constexpr int waves(int xk, int wk) { return xk == kBf16 && wk == 4 ? 6 : 0; }

template <int XK, bool PAIR, int FN, int FM, int WN, int WM, int WK, int KS, int NBUF, bool COLS>
__global__ void __launch_bounds__(64 * WN * WM * WK, waves(XK, WK)) mx_tile_kernel(const MxArgs a) {
  using S = MxTile<XK, PAIR, FN, FM, WN, WM, WK, KS, NBUF, COLS>;
  constexpr int TN = S::TN, TM = S::TM, NW = S::NW, NX = S::NX;
  __shared__ __attribute__((aligned(16))) uint8_t lds[S::kLds];

  Tile tile;
  if (!find_tile<TM>(a, TN, &tile)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wm = wave / WN % WM, wk = wave / (WN * WM);
  const int i = lane & 15, g = lane >> 4;
  const int64_t first_row = tile.expert * a.expert_bytes + (int64_t)tile.n0 * a.row_bytes;
  // (gate and up have the same alignment: both start at a 16-byte boundary plus the window)
  const uint32_t w_odd = (uint32_t)(uintptr_t)(a.w + first_row) & 3u;
  const uint8_t *wbase = a.w + first_row - w_odd;
  const uint8_t *wbase2 = PAIR ? a.w2 + first_row - w_odd : nullptr;
  const int rows_left = a.n - tile.n0;

  // This thread's blocks of a stage: row tid / kBlk + kRowStep v of the tile,
  // block tid % kBlk.  Rows past the matrix read its last row (its bytes, wherever a
  // block starts in them), tokens past the tile's end its first token; their sums
  // are not stored.  A stage is a multiple of four blocks and of four rows a step,
  // so a thread's blocks all start at the same byte of their first word.
  const int wblk = tid % S::kBlk, wrow = tid / S::kBlk;
  const uint32_t wfirst = wblk < a.nb ? 17u * (uint32_t)wblk : 0u;
  const uint32_t wphase = (w_odd + (uint32_t)wrow * (uint32_t)a.row_bytes + wfirst) & 3u;
  uint32_t woff[NW];
#pragma unroll
  for (int v = 0; v < NW; ++v)
    woff[v] = (w_odd + (uint32_t)min((wrow + S::kRowStep * v) % TN, rows_left - 1) * (uint32_t)a.row_bytes + wfirst) & ~3u;
  // A piece of x: a block (MXFP4), or a quarter of one (floats).
  const int xblk = XK == kFp4 ? wblk : (tid >> 2) % S::kBlk;
  const int xtok = XK == kFp4 ? wrow : (tid >> 2) / S::kBlk;
  const uint8_t *xp[NX];
  uint32_t xphase[NX];
  // Tiles of few tokens leave out the loads and writes of the tokens past the
  // end (stale LDS reaches only those tokens' sums); larger ones repeat the
  // first token, since a branch there would part the matrix instructions.
  constexpr bool kSkip = TM <= 32;
  uint32_t there = 0;
#pragma unroll
  for (int v = 0; v < NX; ++v) {
    const int tok = xtok + S::kTokStep * v;
    const int p = tile.m0 + tok < tile.m_end ? tile.m0 + tok : tile.m0;
    there |= (uint32_t)(tok < TM && tile.m0 + tok < tile.m_end) << v;
    int src = p;
    if (a.slots) {
      const int s = a.slots[p];
      src = s < 0 ? -1 : s / a.n_sel;
    }
    if (src < 0 || src >= a.x_rows) src = 0;  // (its outputs are zeros: see the end)
    const uint8_t *row = a.x + src * a.x_bytes;
    if constexpr (XK == kFp4) {  // the first word of this thread's block, and its phase
      row += wfirst;
      xphase[v] = (uint32_t)(uintptr_t)row & 3u;
      row -= xphase[v];
    }
    xp[v] = row;
  }

  // The blocks and pieces of x of the next stage, one by one: piece v < NW is
  // a block of W, the others of x.  Blocks past the row's end are read from an
  // earlier place and zeroed in LDS (TAIL: the row's last stage alone).
  BlockRaw wr[NW], xr4[XK == kFp4 ? NX : 1];
  constexpr int XF = XK == kFp4 ? kBf16 : XK;
  XRaw<XF> xr[XK == kFp4 ? 1 : NX];
  auto fetch = [&](auto piece, int b0) {
    constexpr int v = decltype(piece)::value;
    const uint32_t wb = b0 + wblk < a.nb ? 17u * (uint32_t)b0 : 0u;
    if (kSkip && v >= NW && !(there >> (v < NW ? 0 : v - NW) & 1)) return;
    if constexpr (v < NW) {
      block_load(((PAIR && S::kRowStep * v >= TN) ? wbase2 : wbase) + (woff[v] + wb), wr[v]);
    } else if constexpr (XK == kFp4) {
      block_load(xp[v - NW] + wb, xr4[v - NW]);
    } else {
      constexpr int ES = XK == kF32 ? 4 : 2;
      x_load<XF>(xp[v - NW] + ES * 32u * (uint32_t)min(b0 + xblk, a.nb - 1), xr[v - NW]);
    }
  };
  uint8_t *const cw = lds + (wblk >> 2) * S::kWGroup + 16 * (wblk & 3) + 64 * wrow;
  uint8_t *const cx =
      XK == kFp4 ? lds + S::kOffX + (wblk >> 2) * S::kXGroup + 16 * (wblk & 3) + 64 * wrow
                 : lds + S::kOffX + (xblk >> 2) * S::kXGroup + x_word<XK>(tid & 3) * S::kPlane + 16 * (xblk & 3);
  uint8_t *const sw = lds + S::kOffWS + (wblk >> 2) * S::kWSGroup + 4 * (wblk & 3);
  uint8_t *const sx = lds + S::kOffXS + (wblk >> 2) * S::kXSGroup + 4 * (wblk & 3);
  auto stage = [&](auto piece, auto tail, int b0, int half) {
    constexpr int v = decltype(piece)::value;
    constexpr bool TAIL = decltype(tail)::value;
    const int off = half * S::kStage;
    if (kSkip && v >= NW && !(there >> (v < NW ? 0 : v - NW) & 1)) return;
    if constexpr (v < NW || XK == kFp4) {
      constexpr bool W = v < NW;
      constexpr int j = W ? v : v - NW;
      const int row = wrow + S::kRowStep * j;
      if (!W && TM % S::kRowStep != 0 && row >= TM) return;
      const BlockRaw &r = W ? wr[W ? j : 0] : xr4[W ? 0 : j];
      const uint32_t phase = W ? wphase : xphase[W ? 0 : j];
      u32x4 codes = block_codes(r, phase);
      uint32_t scale = block_scale(r, phase);
      if (TAIL && b0 + wblk >= a.nb) {
        codes = u32x4{0, 0, 0, 0};
        scale = 127;
      }
      *(u32x4 *)((W ? cw : cx) + off + 64 * S::kRowStep * j) = codes;
      ((W ? sw : sx) + off)[256 * (row >> 6) + 16 * (row & 15) + ((row >> 4) & 3)] = (uint8_t)scale;
    } else {
      constexpr int j = v - NW;
      const int tok = xtok + S::kTokStep * j;
      if (TM % S::kTokStep != 0 && tok >= TM) return;
      if (TAIL && b0 + xblk >= a.nb) xr[j] = {};
      u32x4 t[XF];
      x_terms<XF>(xr[j], t);
#pragma unroll
      for (int k = 0; k < XF; ++k) {
        const int col = COLS ? XF * tok + k : tok;
        *(u32x4 *)(cx + off + (COLS ? 0 : k * KS * S::kXGroup) + (col >> 4) * S::kXFrag + 64 * (col & 15)) = t[k];
      }
    }
  };
  constexpr int P = NW + NX;

  f32x4 acc[S::kMats][FN][FM];
#pragma unroll
  for (int u = 0; u < S::kMats; ++u)
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int m = 0; m < FM; ++m) acc[u][n][m] = f32x4{0, 0, 0, 0};

  const int at = 16 * (4 * i + g);  // this lane's piece of a fragment
  // One stage's products in kSlots parts, with between(part) after each: the
  // loads and LDS writes of the stages to come are spread over them, since
  // issued together they hold every wave while the matrix cores idle.
  constexpr int kParts = XK == kFp4 ? FM : 4, kSlots = KS / WK * kParts;
  auto multiply = [&](int half, auto between) {
    const uint8_t *buf = lds + half * S::kStage;
    each<KS / WK>([&](auto kk_) {
      constexpr int kk = decltype(kk_)::value;
      const int grp = wk + WK * kk;
      u32x4 wc[S::kMats][FN];
      uint32_t ws[S::kMats][FN];
#pragma unroll
      for (int u = 0; u < S::kMats; ++u)
#pragma unroll
        for (int n = 0; n < FN; ++n) {
          const int f = u * (TN / 16) + wn * FN + n;  // fragment of the tile
          wc[u][n] = *(const u32x4 *)(buf + grp * S::kWGroup + 1024 * f + at);
          ws[u][n] = *(const uint32_t *)(buf + S::kOffWS + grp * S::kWSGroup + 256 * (f >> 2) + (at >> 2)) >>
                     (8 * (f & 3));
        }
      // x of the part after the current one is read ahead of the LDS writes
      // between the parts.
      const uint8_t *bx = buf + S::kOffX + grp * S::kXGroup + at;
      u32x4 xc[2];
      uint32_t xs[2];
      bf16x8 xb[2][XK == kFp4 ? 1 : FM][S::kTerms];
      auto read_x = [&](auto part_) {
        constexpr int part = decltype(part_)::value;
        if constexpr (XK == kFp4) {
          const int f = wm * FM + part;
          xc[part & 1] = *(const u32x4 *)(bx + 1024 * f);
          xs[part & 1] =
              *(const uint32_t *)(buf + S::kOffXS + grp * S::kXSGroup + 256 * (f >> 2) + (at >> 2)) >> (8 * (f & 3));
        } else {
#pragma unroll
          for (int m = 0; m < FM; ++m)
#pragma unroll
            for (int k = 0; k < S::kTerms; ++k)
              xb[part & 1][XK == kFp4 ? 0 : m][k] =
                  *(const bf16x8 *)(bx + k * KS * S::kXGroup + (wm * FM + m) * S::kXFrag + part * S::kPlane);
        }
      };
      read_x(std::integral_constant<int, 0>());
      each<kParts>([&](auto part_) {
        constexpr int part = decltype(part_)::value;
        if constexpr (part + 1 < kParts) read_x(std::integral_constant<int, part + 1>());
        if constexpr (XK == kFp4) {
          const u32x4 c = xc[part & 1];
          const i32x8 B = {(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
#pragma unroll
          for (int u = 0; u < S::kMats; ++u)
#pragma unroll
            for (int n = 0; n < FN; ++n) {
              const i32x8 A = {(int)wc[u][n].x, (int)wc[u][n].y, (int)wc[u][n].z, (int)wc[u][n].w, 0, 0, 0, 0};
              acc[u][n][part] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, acc[u][n][part], 4, 4, 0,
                                                                                 (int)ws[u][n], 0, (int)xs[part & 1]);
            }
        } else {
#pragma unroll
          for (int u = 0; u < S::kMats; ++u)
#pragma unroll
            for (int n = 0; n < FN; ++n) {
              const bf16x8 A = weights8(wc[u][n][part], scale_of(ws[u][n], 0));
#pragma unroll
              for (int m = 0; m < FM; ++m)
#pragma unroll
                for (int k = 0; k < S::kTerms; ++k)
                  acc[u][n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, xb[part & 1][m][k], acc[u][n][m], 0, 0, 0);
            }
        }
        between(std::integral_constant<int, kk * kParts + part>());
      });
    });
  };
  // The pieces of one part: all P spread over the kSlots parts.
  auto pieces = [&](auto slot, auto f) {
    constexpr int s = decltype(slot)::value, p0 = s * P / kSlots, p1 = (s + 1) * P / kSlots;
    each<p1 - p0>([&](auto q) { f(std::integral_constant<int, p0 + decltype(q)::value>()); });
  };
  const std::true_type last;
  const std::false_type inner;

  const int stages = (a.nb + S::kBlk - 1) / S::kBlk;
  if (stages > 0) {
    each<P>([&](auto p) { fetch(p, 0); });
    int t = 0;
    if constexpr (NBUF == 2) {
      // stage t + 1 goes from registers to LDS, and t + 2 into the registers,
      // while t is multiplied
      each<P>([&](auto p) { stage(p, last, 0, 0); });
      if (S::kOneLoop || stages > 1) each<P>([&](auto p) { fetch(p, S::kBlk); });
      __syncthreads();
      if constexpr (S::kOneLoop) {
        // The last two stages in the same code as the others: loads past the
        // row's end read its first blocks, and what they put into LDS is not
        // multiplied.  Code of their own, below, leaves no register free and
        // spills (4096 x 24576 products of k = 6144: 598 us, 386 so), but
        // where it fits saves those loads and the checks (4 x 4 fragments of a
        // wave: 463 us, 513 so).
        for (; t < stages; ++t) {
          multiply(t & 1, [&](auto slot) {
            pieces(slot, [&](auto p) {
              stage(p, last, (t + 1) * S::kBlk, (t + 1) & 1);
              fetch(p, (t + 2) * S::kBlk);
            });
          });
          __syncthreads();
        }
      }
      for (; t + 2 < stages; ++t) {
        multiply(t & 1, [&](auto slot) {
          pieces(slot, [&](auto p) {
            stage(p, inner, (t + 1) * S::kBlk, (t + 1) & 1);
            fetch(p, (t + 2) * S::kBlk);
          });
        });
        __syncthreads();
      }
      for (; t < stages; ++t) {
        multiply(t & 1, [&](auto slot) {
          if (t + 1 < stages) pieces(slot, [&](auto p) { stage(p, last, (t + 1) * S::kBlk, (t + 1) & 1); });
        });
        __syncthreads();
      }
    } else {
      for (; t + 1 < stages; ++t) {
        each<P>([&](auto p) { stage(p, inner, t * S::kBlk, 0); });
        __syncthreads();
        multiply(0, [&](auto slot) { pieces(slot, [&](auto p) { fetch(p, (t + 1) * S::kBlk); }); });
        __syncthreads();
      }
      each<P>([&](auto p) { stage(p, last, t * S::kBlk, 0); });
      __syncthreads();
      multiply(0, [](auto) {});
      if (WK > 1) __syncthreads();
    }
  }

  if constexpr (WK > 1) {
    // the other waves' sums to the first of each tile part, added in their order
    f32x4 *red = (f32x4 *)lds + (wm * WN + wn) * S::kMats * FN * FM * 64 + lane;
    constexpr int kPart = WN * WM * S::kMats * FN * FM * 64;
#pragma unroll
    for (int u = 0; u < S::kMats; ++u)
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int m = 0; m < FM; ++m)
          if (wk > 0) red[(wk - 1) * kPart + ((u * FN + n) * FM + m) * 64] = acc[u][n][m];
    __syncthreads();
    if (wk > 0) return;
#pragma unroll
    for (int u = 0; u < S::kMats; ++u)
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
          for (int w = 0; w < WK - 1; ++w) acc[u][n][m] += red[w * kPart + ((u * FN + n) * FM + m) * 64];
  }

  if constexpr (COLS) {
    // a token's columns to its first one, the largest term first
#pragma unroll
    for (int u = 0; u < S::kMats; ++u)
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = acc[u][n][0][e];
          float sum = v + __shfl_down(v, 1);
          if constexpr (S::kCols == 3) sum += __shfl_down(v, 2);
          acc[u][n][0][e] = sum;
        }
  }
  // The outputs of fragment (n, m): four of consecutive n for this lane's token.
  auto outputs = [&](int n, int m) {
    f32x4 v = acc[0][n][m];
    if constexpr (PAIR)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = silu_times(v[e], acc[S::kMats - 1][n][m][e]);
    return v;
  };
  // a place whose source x does not have
  auto absent = [&](int p) {
    return a.slots && (uint32_t)(a.slots[p] < 0 ? -1 : a.slots[p] / a.n_sel) >= (uint32_t)a.x_rows;
  };
  // the place of this lane's token m, or one past the tile's end
  auto place = [&](int m) {
    if (COLS) return i % S::kCols == 0 && i / S::kCols < TM ? tile.m0 + i / S::kCols : tile.m_end;
    return tile.m0 + 16 * (wm * FM + m) + i;
  };
  // Rows (bits of each fragment) whose sums of every token of this wave are
  // infinities or NaN.  First whether there is any such sum at all (or products
  // of sums past fp32's range, which are looked through for nothing): a tile of
  // ordinary numbers pays no more.
  uint32_t odd[FN] = {}, any_odd = 0;
  if constexpr (XK != kFp4) {
    auto sums = [&](auto ragged) {  // (rows past the matrix hold anything)
      float all = 0.0f;
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        float some = 0.0f;
#pragma unroll
        for (int u = 0; u < S::kMats; ++u)
#pragma unroll
          for (int n = 0; n < FN; ++n) {
            f32x4 v = acc[u][n][m];
            if constexpr (decltype(ragged)::value)
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = 16 * (wn * FN + n) + 4 * g + e < rows_left ? v[e] : 0.0f;
            some = fmaf(v.x, v.y, fmaf(v.z, v.w, some));
          }
        if (place(m) < tile.m_end) all += some;
      }
      return all;
    };
    const float all = rows_left < TN ? sums(std::true_type()) : sums(std::false_type());
    if (__builtin_expect(__ballot(!__builtin_isfinite(all)) != 0, 0)) {
#pragma unroll
      for (int n = 0; n < FN; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          bool finite = false;
#pragma unroll
          for (int m = 0; m < FM; ++m)
            finite |= place(m) < tile.m_end && __builtin_isfinite(acc[0][n][m][e]) &&
                      (!PAIR || __builtin_isfinite(acc[S::kMats - 1][n][m][e]));
          const uint64_t lanes = __ballot(finite);
#pragma unroll
          for (int r = 0; r < 4; ++r) odd[n] |= (lanes >> (16 * r) & 0xffffu ? 0u : 1u) << (4 * r + e);
        }
        any_odd |= odd[n];
      }
    }
  }
  if constexpr (S::kRows) {
    if (a.y_type == QG_F32) store_rows<S, 4>(a, tile, lds, wn, wm, i, g, outputs, absent);
    else store_rows<S, 2>(a, tile, lds, wn, wm, i, g, outputs, absent);
    if (XK != kFp4) __syncthreads();  // (other waves have stored these outputs)
  } else {
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      const int p = place(m);
      if (p >= tile.m_end) continue;
      const bool none = absent(p);
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        const int r = tile.n0 + 16 * (wn * FN + n) + 4 * g;
        const f32x4 v = outputs(n, m);
        if (r < a.n) store4(a, p, r, a.n - r, none ? f32x4{0, 0, 0, 0} : v);
      }
    }
  }
  if constexpr (XK != kFp4) {
    // Weights of 2^128 and more were infinities above, so every token's sum of
    // their row is one or NaN: such rows are found among those, and computed
    // again, one output a lane.  (No quantisation of fp32 values writes such
    // scales.  333 bf16 tokens, 11008-row pair of k = 4096: 84 us, as many with a
    // token of NaN, 133 with all tokens NaN, 370 with one large row; 80 products
    // of ordinary values take 1.005 times what they do without the check.)
    if (__builtin_expect(!any_odd, 1)) return;
    constexpr int kTokens = COLS ? TM : 16 * FM;  // of this wave
    const int p0 = tile.m0 + (COLS ? 0 : 16 * FM * wm), p1 = min(p0 + kTokens, tile.m_end);
    if (p0 >= p1) return;
    // (lane and address anew: kept from the start they would cost the main loop registers)
    const int64_t first = tile.expert * a.expert_bytes + (int64_t)__builtin_amdgcn_readfirstlane(tile.n0) * a.row_bytes;
    const uint8_t *w = a.w + first, *w2 = PAIR ? a.w2 + first : nullptr;
    const int here = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
#pragma unroll 1
    for (int n = 0; n < FN; ++n) {
      uint32_t rows = odd[0];
#pragma unroll
      for (int j = 1; j < FN; ++j) rows = n == j ? odd[j] : rows;
      const int r0 = 16 * (wn * FN + n), row = r0 + (here & 15);
      const bool look = row < rows_left && (rows >> (here & 15) & 1);
      const int64_t at_row = (int64_t)row * a.row_bytes;
      bool large = false, huge = false;
      if (look)
#pragma unroll 4
        for (int b = here >> 4; b < a.nb; b += 4) {
          const int e = w[at_row + 17 * b], e2 = PAIR ? w2[at_row + 17 * b] : 0;
          large |= e == 253 || e == 254 || e2 == 253 || e2 == 254;
        }
      if (large)
#pragma unroll 1
        for (int b = here >> 4; b < a.nb; b += 4)
          huge |= huge_block(w + at_row + 17 * b) || (PAIR && huge_block(w2 + at_row + 17 * b));
      const uint64_t lanes = __ballot(huge);
      rows = (uint32_t)(lanes | lanes >> 16 | lanes >> 32 | lanes >> 48) & 0xffffu;
      for (; rows; rows &= rows - 1) {
        const int r = r0 + __builtin_ctz(rows);
#pragma unroll 1
        for (int p = p0 + here; p < p1; p += 64) {
          if (absent(p)) continue;
          const uint8_t *x = a.x + (int64_t)(a.slots ? a.slots[p] / a.n_sel : p) * a.x_bytes;
          float v = one_output<XK>(w + (int64_t)r * a.row_bytes, x, a.nb);
          if (PAIR) v = silu_times(v, one_output<XK>(w2 + (int64_t)r * a.row_bytes, x, a.nb));
          store4(a, p, tile.n0 + r, 1, f32x4{v, 0, 0, 0});
        }
      }
    }
  }
}

// Tiles along the rows of W, and all of the grid.
template <typename S>
struct Grid {
  int64_t tn, all;
  explicit Grid(const MxArgs &a) {
    tn = ((int64_t)a.n + S::TN - 1) / S::TN;
    // experts: a partial tile each beyond the whole ones, as far as places go
    const int64_t tm = a.offsets ? a.places / S::TM + (int64_t)(a.n_expert < a.places ? a.n_expert : a.places)
                                 : ((int64_t)a.places + S::TM - 1) / S::TM;
    all = tn * tm;
  }
  // a grid holds fewer than 2^32 threads
  bool fits() const { return all < (1ll << 32) / S::kThreads - 8; }
};

template <int XK, bool PAIR, int FN, int FM, int WN, int WM, int WK, int KS, int NBUF, bool COLS = false>
hipError_t launch_tile(MxArgs a, hipStream_t stream) {
  using S = MxTile<XK, PAIR, FN, FM, WN, WM, WK, KS, NBUF, COLS>;
  const Grid<S> grid(a);
  a.tiles_n = (int)grid.tn;
  a.tiles = (int)grid.all;
  hipLaunchKernelGGL((mx_tile_kernel<XK, PAIR, FN, FM, WN, WM, WK, KS, NBUF, COLS>),
                     dim3((unsigned)((grid.all + 7) / 8 * 8)), dim3(S::kThreads), 0, stream, a);
  return hipGetLastError();
}

// The variants of one activation kind (one translation unit each).  *fits:
// false, and nothing launched, if no variant's grid holds the product.
template <int XK> hipError_t launch_mx(const MxArgs &a, hipStream_t stream, bool *fits);

}  // namespace qgemv_mx
