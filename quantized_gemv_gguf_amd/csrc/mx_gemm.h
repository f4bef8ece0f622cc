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
//             product is exact and only the fp32 sums round.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

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

// Tile `id` of the grid.  Workgroups go to the eight XCDs in turn; each XCD
// takes one contiguous run of tiles, so that neighbours in the order below
// share an L2.  Order: experts; within an expert bands of eight token tiles;
// within a band tile rows n, and innermost the band's token tiles, so one
// weight tile is read by up to eight neighbours and the band's tokens stay in
// the XCD's L2 for the whole sweep over n.
// Every wave finds its tile by itself: lane l sums the token tiles of its run
// of experts, a scan over the lanes gives the first tile of each run, and the
// lane whose run holds the tile walks it.
template <int TM>
__device__ __forceinline__ bool find_tile(const MxArgs &a, int tn_rows, Tile *t) {
  const int per = (a.tiles + 7) >> 3;
  const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || id >= a.tiles) return false;
  int e = 0, lo = 0, hi = a.places, rem = id;
  if (a.offsets) {
    const int lane = threadIdx.x & 63;
    const int run = (a.n_expert + 63) >> 6;
    const int e0 = min(lane * run, a.n_expert), e1 = min(e0 + run, a.n_expert);
    auto at = [&](int i) { return min(max(a.offsets[i], 0), a.places); };
    int mine = 0, o = e0 < e1 ? at(e0) : 0;
    for (int i = e0; i < e1; ++i) {
      const int q = at(i + 1);
      mine += (max(q - o, 0) + TM - 1) / TM;
      o = q;
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    const int mt = id / a.tiles_n;  // token tiles before this tile's expert's end
    const uint64_t past = __ballot(upto > mt);
    if (!past) return false;        // behind the last expert's last tile
    const int src = __builtin_ctzll(past);
    int first = __shfl(upto - mine, src);
    e = __shfl(e0, src);
    const int last = __shfl(e1, src);
    lo = at(e);
    hi = at(e + 1);
    for (;;) {
      const int tiles = (max(hi - lo, 0) + TM - 1) / TM;
      if (mt < first + tiles || e + 1 >= last) break;
      first += tiles;
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

// The bf16 terms of eight values in the lane order of the codes' word: element
// pairs (lo[b], hi[b]), lo = four values from 4q, hi = four from 16 + 4q.
// Terms are cut, not rounded: the rest is exact, and an infinity or NaN stays
// in the first term alone.
template <int XK> struct XRaw;
template <> struct XRaw<kBf16> { u32x2 lo, hi; };
template <> struct XRaw<kF16> { u32x2 lo, hi; };
template <> struct XRaw<kF32> { f32x4 lo, hi; };

__device__ __forceinline__ uint32_t top_halves(uint32_t lo, uint32_t hi) {  // (lo >> 16) | (hi & 0xffff0000)
  return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

// v cut to its first bf16; *rest = v minus it, exactly (0 for an infinity or NaN)
__device__ __forceinline__ uint32_t cut(float v, float *rest) {
  const uint32_t b = __float_as_uint(v);
  const bool fine = (b & 0x7f800000u) != 0x7f800000u;
  // a NaN keeps a set top mantissa bit, so the cut does not turn it into an infinity
  const uint32_t h = (b & 0xffff0000u) | (v != v ? 0x00400000u : 0u);
  *rest = fine ? v - __uint_as_float(h) : 0.0f;
  return h;
}

template <int XK>
__device__ __forceinline__ void x_terms(const XRaw<XK> &r, u32x4 (&out)[XK]) {
  if constexpr (XK == kBf16) {
    out[0] = u32x4{__builtin_amdgcn_perm(r.hi.x, r.lo.x, 0x05040100u), __builtin_amdgcn_perm(r.hi.x, r.lo.x, 0x07060302u),
                   __builtin_amdgcn_perm(r.hi.y, r.lo.y, 0x05040100u), __builtin_amdgcn_perm(r.hi.y, r.lo.y, 0x07060302u)};
  } else {
    float lo[4], hi[4];
    if constexpr (XK == kF16) {
      typedef _Float16 h4 __attribute__((ext_vector_type(4)));
      const h4 l = __builtin_bit_cast(h4, r.lo), h = __builtin_bit_cast(h4, r.hi);
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
          const uint32_t l = cut(lo[b], &rl), h = cut(hi[b], &rh);
          out[t][b] = top_halves(l, h);
          lo[b] = rl;
          hi[b] = rh;
        }
      }
  }
}

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

// The tiled product.  A workgroup of WN x WM waves owns 16 FN WN rows of W (of
// each of a pair) and 16 FM WM tokens; a wave 16 FN x 16 FM.  Per step of four
// blocks (128 values): the next step's blocks and activations are loaded into
// registers while the current step, in LDS, is multiplied.
// LDS: codes row-major, 16 bytes per (row, block), so a wave's fragment of 16
// rows is 1 KB read once without conflicts; scale bytes of four fragments of
// 16 rows in one word; float x as [term][fragment][word j][token][block], one
// fragment and word 1 KB in a row, planes of words 64 bytes apart beyond it so
// that a token's sixteen pieces are written to sixteen bank groups.
template <int XK, bool PAIR, int FN, int FM, int WN, int WM>
struct MxTile {
  static constexpr int kThreads = 64 * WN * WM;
  static constexpr int TN = 16 * FN * WN, TM = 16 * FM * WM;
  static constexpr int kMats = PAIR ? 2 : 1;
  static constexpr int kWRows = TN * kMats;
  static constexpr int NW = kWRows * 4 / kThreads;                          // blocks of W per thread and step
  static constexpr int NX = XK == kFp4 ? (TM * 4 + kThreads - 1) / kThreads : (TM * 16 + kThreads - 1) / kThreads;
  static constexpr int kPlane = 1024 + 64;                                   // one word of 16 tokens, padded
  static constexpr int kXFrag = 4 * kPlane;
  static constexpr int kWBytes = kWRows * 64, kWScale = kWRows * 4;
  static constexpr int kXBytes = XK == kFp4 ? TM * 64 : XK * (TM / 16) * kXFrag;
  static constexpr int kXScale = XK == kFp4 ? (TM + 63) / 64 * 256 : 0;
  static constexpr int kLds = kWBytes + kWScale + kXBytes + kXScale;
  static_assert(kWRows * 4 % kThreads == 0 && kThreads == 256, "a step's blocks divide over 256 threads");
};

template <int XK, bool PAIR, int FN, int FM, int WN, int WM>
__global__ void __launch_bounds__(256) mx_tile_kernel(const MxArgs a) {
  using S = MxTile<XK, PAIR, FN, FM, WN, WM>;
  constexpr int TN = S::TN, TM = S::TM, NW = S::NW, NX = S::NX;
  __shared__ __attribute__((aligned(16))) uint8_t lds[S::kLds];
  uint8_t *lw = lds, *lws = lds + S::kWBytes, *lx = lws + S::kWScale, *lxs = lx + S::kXBytes;

  Tile tile;
  if (!find_tile<TM>(a, TN, &tile)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wm = wave / WN;
  const int i = lane & 15, g = lane >> 4;
  const uint8_t *wbase = a.w + tile.expert * a.expert_bytes + (int64_t)tile.n0 * a.row_bytes;
  const uint8_t *wbase2 = PAIR ? a.w2 + tile.expert * a.expert_bytes + (int64_t)tile.n0 * a.row_bytes : nullptr;
  const int rows_left = a.n - tile.n0;

  // This thread's blocks of a step: row (tid / 4 + 64 v) of the tile, block
  // tid % 4.  Rows past the matrix read its last row; their sums are not stored.
  uint32_t woff[NW];
#pragma unroll
  for (int v = 0; v < NW; ++v) {
    const int row = (tid >> 2) + 64 * v;
    woff[v] = (uint32_t)min(row % TN, rows_left - 1) * (uint32_t)a.row_bytes + 17u * (tid & 3);
  }
  // This thread's rows of x: null for places past the tile's end and sources
  // x does not have, which count as zeros.
  const uint8_t *xp[NX];
#pragma unroll
  for (int v = 0; v < NX; ++v) {
    const int tok = XK == kFp4 ? (tid >> 2) + 64 * v : (tid >> 4) + 16 * v;
    const int p = tile.m0 + tok;
    xp[v] = nullptr;
    if (tok < TM && p < tile.m_end) {
      int src = p;
      if (a.slots) {
        const int s = a.slots[p];
        src = s < 0 ? -1 : s / a.n_sel;
      }
      if (src >= 0 && src < a.x_rows) xp[v] = a.x + src * a.x_bytes;
    }
  }

  u32x4 wr[NW];
  uint32_t wsr[NW];
  u32x4 xr4[NX];
  uint32_t xsr[NX];
  XRaw<XK == kFp4 ? kBf16 : XK> xr[NX];
  auto fetch = [&](int b0) {
    const bool wok = b0 + (tid & 3) < a.nb;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      const uint8_t *base = (PAIR && 64 * v >= TN) ? wbase2 : wbase;  // 64 divides TN
      wr[v] = u32x4{0, 0, 0, 0};
      wsr[v] = 127;
      if (wok) {
        const uint8_t *p = base + (woff[v] + 17u * (uint32_t)b0);
        __builtin_memcpy(&wr[v], p + 1, 16);
        wsr[v] = p[0];
      }
    }
    if constexpr (XK == kFp4) {
#pragma unroll
      for (int v = 0; v < NX; ++v) {
        xr4[v] = u32x4{0, 0, 0, 0};
        xsr[v] = 127;
        if (wok && xp[v]) {
          const uint8_t *p = xp[v] + 17u * (uint32_t)(b0 + (tid & 3));
          __builtin_memcpy(&xr4[v], p + 1, 16);
          xsr[v] = p[0];
        }
      }
    } else {
      constexpr int ES = XK == kF32 ? 4 : 2;
      const int blk = (tid >> 2) & 3, q = tid & 3;
      const bool ok = b0 + blk < a.nb;
#pragma unroll
      for (int v = 0; v < NX; ++v) {
        xr[v] = {};
        if (ok && xp[v]) {
          const uint8_t *p = xp[v] + (uint32_t)ES * (32u * (uint32_t)(b0 + blk) + 4u * q);
          __builtin_memcpy(&xr[v].lo, p, 4 * ES);
          __builtin_memcpy(&xr[v].hi, p + 16 * ES, 4 * ES);
        }
      }
    }
  };
  auto stage = [&]() {
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      *(u32x4 *)(lw + 16 * (tid + 256 * v)) = wr[v];
      lws[256 * v + 4 * (tid & 63) + (tid >> 6)] = (uint8_t)wsr[v];
    }
    if constexpr (XK == kFp4) {
#pragma unroll
      for (int v = 0; v < NX; ++v)
        if ((tid >> 2) + 64 * v < TM) {
          *(u32x4 *)(lx + 16 * (tid + 256 * v)) = xr4[v];
          lxs[256 * v + 4 * (tid & 63) + (tid >> 6)] = (uint8_t)xsr[v];
        }
    } else {
      const int blk = (tid >> 2) & 3, q = tid & 3;
#pragma unroll
      for (int v = 0; v < NX; ++v)
        if ((tid >> 4) + 16 * v < TM) {
          u32x4 t[XK];
          x_terms<XK>(xr[v], t);
#pragma unroll
          for (int k = 0; k < XK; ++k)
            *(u32x4 *)(lx + (k * (TM / 16) + v) * S::kXFrag + q * S::kPlane + ((tid >> 4) * 4 + blk) * 16) = t[k];
        }
    }
  };

  f32x4 acc[S::kMats][FN][FM];
#pragma unroll
  for (int u = 0; u < S::kMats; ++u)
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int m = 0; m < FM; ++m) acc[u][n][m] = f32x4{0, 0, 0, 0};

  fetch(0);
  for (int b0 = 0; b0 < a.nb; b0 += 4) {
    stage();
    __syncthreads();
    if (b0 + 4 < a.nb) fetch(b0 + 4);
    u32x4 wc[S::kMats][FN];
    uint32_t ws[S::kMats][FN];
#pragma unroll
    for (int u = 0; u < S::kMats; ++u)
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        const int f = u * (TN / 16) + wn * FN + n;  // fragment of the tile
        wc[u][n] = *(const u32x4 *)(lw + 1024 * f + 16 * (4 * i + g));
        ws[u][n] = *(const uint32_t *)(lws + 256 * (f >> 2) + 4 * (4 * i + g)) >> (8 * (f & 3));
      }
    if constexpr (XK == kFp4) {
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        const int f = wm * FM + m;
        const u32x4 xc = *(const u32x4 *)(lx + 1024 * f + 16 * (4 * i + g));
        const uint32_t xs = *(const uint32_t *)(lxs + 256 * (f >> 2) + 4 * (4 * i + g)) >> (8 * (f & 3));
        const i32x8 B = {(int)xc.x, (int)xc.y, (int)xc.z, (int)xc.w, 0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < S::kMats; ++u)
#pragma unroll
          for (int n = 0; n < FN; ++n) {
            const i32x8 A = {(int)wc[u][n].x, (int)wc[u][n].y, (int)wc[u][n].z, (int)wc[u][n].w, 0, 0, 0, 0};
            acc[u][n][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, acc[u][n][m], 4, 4, 0,
                                                                            (int)ws[u][n], 0, (int)xs);
          }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf16x8 xb[FM][XK];
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
          for (int k = 0; k < XK; ++k)
            xb[m][k] = *(const bf16x8 *)(lx + (k * (TM / 16) + wm * FM + m) * S::kXFrag + j * S::kPlane +
                                         16 * (4 * i + g));
#pragma unroll
        for (int u = 0; u < S::kMats; ++u)
#pragma unroll
          for (int n = 0; n < FN; ++n) {
            const bf16x8 A = weights8(wc[u][n][j], scale_of(ws[u][n], 0));
#pragma unroll
            for (int m = 0; m < FM; ++m)
#pragma unroll
              for (int k = 0; k < XK; ++k)
                acc[u][n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, xb[m][k], acc[u][n][m], 0, 0, 0);
          }
      }
    }
    __syncthreads();
  }

#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const int p = tile.m0 + 16 * (wm * FM + m) + i;
    if (p >= tile.m_end) continue;
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      const int r = tile.n0 + 16 * (wn * FN + n) + 4 * g;
      f32x4 v = acc[0][n][m];
      if constexpr (PAIR)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = silu_times(v[e], acc[1][n][m][e]);
      if (r < a.n) store4(a, p, r, a.n - r, v);
    }
  }
}

template <int XK, bool PAIR, int FN, int FM, int WN, int WM>
hipError_t launch_tile(MxArgs a, hipStream_t stream) {
  using S = MxTile<XK, PAIR, FN, FM, WN, WM>;
  const int64_t tn = ((int64_t)a.n + S::TN - 1) / S::TN;
  // experts: a partial tile each beyond the whole ones, as far as places go
  const int64_t tm = a.offsets ? a.places / S::TM + (int64_t)(a.n_expert < a.places ? a.n_expert : a.places)
                               : ((int64_t)a.places + S::TM - 1) / S::TM;
  if (tn * tm > 0x7ffffff0) return hipErrorInvalidConfiguration;
  a.tiles_n = (int)tn;
  a.tiles = (int)(tn * tm);
  hipLaunchKernelGGL((mx_tile_kernel<XK, PAIR, FN, FM, WN, WM>), dim3((unsigned)((tn * tm + 7) / 8 * 8)), dim3(256), 0,
                     stream, a);
  return hipGetLastError();
}

// The variants of one activation kind (one translation unit each).
template <int XK> hipError_t launch_mx(const MxArgs &a, hipStream_t stream);

}  // namespace qgemv_mx
