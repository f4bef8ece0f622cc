// mx.hip -- the C ABI of include/qgemv_mx.h, with quantisation to MXFP4 and the
// routing kernels (sort by expert, gather, weighted sum back, its gradient).
// The products' kernels are in mx_gemm.h.
#include "mx_gemm.h"

#include <algorithm>
#include <type_traits>

namespace qgemv_detail {
int record_hip_error(hipError_t e, const char *what);  // qgemv.hip: for qgemv_last_hip_error
}

using namespace qgemv_mx;

namespace {

// ---------------------------------------------------------------------------
// Element types
// ---------------------------------------------------------------------------

template <int T> struct Elem;
template <> struct Elem<QG_F32> {
  typedef float Raw;
  static constexpr int kSize = 4;
  __device__ static inline float to(Raw v) { return v; }
  __device__ static inline Raw from(float v) { return v; }
};
template <> struct Elem<QG_F16> {
  typedef _Float16 Raw;
  static constexpr int kSize = 2;
  __device__ static inline float to(Raw v) { return (float)v; }
  __device__ static inline Raw from(float v) { return (_Float16)v; }
};
template <> struct Elem<QG_BF16> {
  typedef __bf16 Raw;
  static constexpr int kSize = 2;
  __device__ static inline float to(Raw v) { return (float)v; }
  __device__ static inline Raw from(float v) { return (__bf16)v; }
};

typedef u32x4 __attribute__((aligned(2))) u32x4_2;  // 16 bytes at any element

// N values from / to any element-aligned address, as one access of N elements.
template <int T, int N>
__device__ __forceinline__ void load_n(const void *p, float (&v)[N]) {
  typedef typename Elem<T>::Raw V __attribute__((ext_vector_type(N)));
  V r;
  __builtin_memcpy(&r, p, N * Elem<T>::kSize);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = Elem<T>::to(r[i]);
}
template <int T, int N>
__device__ __forceinline__ void store_n(void *p, const float (&v)[N]) {
  typedef typename Elem<T>::Raw V __attribute__((ext_vector_type(N)));
  V r;
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = Elem<T>::from(v[i]);
  __builtin_memcpy(p, &r, N * Elem<T>::kSize);
}

// ---------------------------------------------------------------------------
// Quantisation.  Four lanes per block of 32: lane q holds elements 4q + b and
// 16 + 4q + b (b < 4), which are word q of the block's codes.  Bound by memory:
// one pass, the 17-byte blocks put together in LDS so that they are written in
// whole granules.  8192 x 6144 bf16: 25.8 us quantised and 19.9 back, 4.9 and
// 6.4 TB/s (a copy: 5.2).
// ---------------------------------------------------------------------------

constexpr int kQBlocks = 256;  // blocks per workgroup: 4352 bytes, 272 granules

// (group0, here and below: the launch's first workgroup of all, see in_grids)

template <int T>
__global__ void __launch_bounds__(256) quantize_kernel(const uint8_t *x, int64_t stride, int nb, int64_t blocks,
                                                       uint8_t *out, int64_t group0) {
  __shared__ __attribute__((aligned(16))) uint8_t buf[kQBlocks * 17];
  constexpr int ES = Elem<T>::kSize;
  const int tid = threadIdx.x, q = tid & 3;
  const int64_t first = (group0 + blockIdx.x) * kQBlocks;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int bl = 64 * v + (tid >> 2);
    const int64_t b = first + bl;
    if (b < blocks) {
      const int64_t r = b / nb;
      const uint8_t *p = x + (r * stride + 32 * (b - r * nb) + 4 * q) * ES;
      float lo[4], hi[4];
      load_n<T>(p, lo);
      load_n<T>(p + 16 * ES, hi);
      // the largest magnitude as bits: their order is the magnitudes' order,
      // infinities and NaN above every finite one
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        m = max(m, __float_as_uint(lo[e]) & 0x7fffffffu);
        m = max(m, __float_as_uint(hi[e]) & 0x7fffffffu);
      }
      m = max(m, (uint32_t)__shfl_xor((int)m, 1));
      m = max(m, (uint32_t)__shfl_xor((int)m, 2));
      // floor(log2 a) - 2 + 127 is the exponent field less 2 for a normal a,
      // and below 0 for a subnormal one
      const int field = (int)(m >> 23);
      const bool fine = field < 255;
      const int e = fine ? max(field - 2, 0) : 255;
      const float scale = __uint_as_float((uint32_t)e << 23);
      uint32_t c = 0;
      if (fine) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, lo[0], hi[0], scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, lo[1], hi[1], scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, lo[2], hi[2], scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, lo[3], hi[3], scale, 3);
      }
      uint8_t *o = buf + 17 * bl;
      if (q == 0) o[0] = (uint8_t)e;
      __builtin_memcpy(o + 1 + 4 * q, &c, 4);
    }
  }
  __syncthreads();
  const int64_t left = min((int64_t)kQBlocks, blocks - first) * 17;  // bytes
  uint8_t *dst = out + first * 17;                                   // 16-byte aligned: 4352 = 16 * 272
  for (int o = 16 * tid; o < left; o += 4096) {
    if (o + 16 <= left) *(u32x4 *)(dst + o) = *(const u32x4 *)(buf + o);
    else
      for (int k = o; k < left; ++k) dst[k] = buf[k];
  }
}

template <int T>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t *w, int nb, int64_t blocks, uint8_t *out,
                                                         int64_t stride, int64_t group0) {
  constexpr int ES = Elem<T>::kSize;
  const int q = threadIdx.x & 3;
  const int64_t b = (group0 + blockIdx.x) * 64 + (threadIdx.x >> 2);
  if (b >= blocks) return;
  const uint8_t *p = w + b * 17;
  uint32_t c;
  __builtin_memcpy(&c, p + 1 + 4 * q, 4);
  const float s = __uint_as_float((uint32_t)p[0] << 23);
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
  const f2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
  const float lo[4] = {v0.x, v1.x, v2.x, v3.x}, hi[4] = {v0.y, v1.y, v2.y, v3.y};
  const int64_t r = b / nb;
  uint8_t *o = out + (r * stride + 32 * (b - r * nb) + 4 * q) * ES;
  store_n<T>(o, lo);
  store_n<T>(o + 16 * ES, hi);
}

// ---------------------------------------------------------------------------
// Routing
// ---------------------------------------------------------------------------

// Workgroup e < n_expert places the slots of expert e: its first pass counts
// the ids below e (the expert's offset) and equal to e per wave, its second
// writes each slot's place, in slot order (a lane's four ids, then the lanes,
// then the groups of 256, then the waves).  Workgroup n_expert does the same
// for the dropped slots: pos -1, and slots -1 behind the last kept one.  No
// atomics, no workspace, one launch; every workgroup reads all ids from L2,
// eight groups of 256 at a time so that their loads overlap (kept in registers
// between the passes where a wave has no more).  32768 slots of 128 experts:
// 8 us, 16 with the loads one by one.
constexpr int kSortWaves = 16, kSortGroups = 8;
__global__ void __launch_bounds__(64 * kSortWaves) sort_kernel(const int32_t *ids, int n, int n_expert,
                                                               int32_t *offsets, int32_t *slots, int32_t *pos) {
  __shared__ int below[kSortWaves], equal[kSortWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.x;
  const int groups = (n + 255) / 256, per = (groups + kSortWaves - 1) / kSortWaves;
  const int g0 = min(wave * per, groups), g1 = min(g0 + per, groups);
  int v[kSortGroups][4];
  auto load = [&](int g) {  // groups g .. g + 7 of the wave; ids past the end are no expert's
#pragma unroll
    for (int j = 0; j < kSortGroups; ++j) {
      const int at = 256 * (g + j) + 4 * lane;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[j][k] = 0x7fffffff;
      if (g + j >= g1) continue;
      if (at + 4 <= n) {
        __builtin_memcpy(v[j], ids + at, 16);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (at + k < n) v[j][k] = ids[at + k];
      }
    }
  };
  // sums of counts up to 32 over the lanes, bit by bit
  auto lanes_sum = [](int c) {
    int sum = 0;
#pragma unroll
    for (int b = 0; b < 6; ++b) sum += __popcll(__ballot(c >> b & 1)) << b;
    return sum;
  };
  int nb = 0, ne = 0;
  for (int g = g0; g < g1; g += kSortGroups) {
    load(g);
    int cb = 0, ce = 0;
#pragma unroll
    for (int j = 0; j < kSortGroups; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        cb += (uint32_t)v[j][k] < (uint32_t)e;
        ce += v[j][k] == e;
      }
    nb += lanes_sum(cb);
    ne += lanes_sum(ce);
  }
  if (lane == 0) {
    below[wave] = nb;
    equal[wave] = ne;
  }
  __syncthreads();
  int base = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    base += below[w];
    if (w < wave) before += equal[w];
  }
  if (threadIdx.x == 0) offsets[e] = base;
  if (e == n_expert) {
    for (int p = base + (int)threadIdx.x; p < n; p += 64 * kSortWaves) slots[p] = -1;
    for (int i = (int)threadIdx.x; i < n; i += 64 * kSortWaves)
      if ((uint32_t)ids[i] >= (uint32_t)n_expert) pos[i] = -1;
    return;
  }
  if (ne == 0) return;
  int at = base + before;
  const uint64_t lower = (1ull << lane) - 1;
  for (int g = g0; g < g1; g += kSortGroups) {
    if (g1 - g0 > kSortGroups) load(g);
#pragma unroll
    for (int j = 0; j < kSortGroups; ++j) {
      uint64_t b[4], any = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) any |= b[k] = __ballot(v[j][k] == e);
      if (!any) continue;
      int rank = at;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        rank += __popcll(b[k] & lower);
        at += __popcll(b[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (v[j][k] != e) continue;
        const int slot = 256 * (g + j) + 4 * lane + k;
        slots[rank] = slot;
        pos[slot] = rank;
        ++rank;
      }
    }
  }
}

// Many slots, in four launches over chunks of at most kChunk slots (and at
// least QG_MAX_EXPERTS), which keep their tables in the outputs:
//   count    a chunk's slots of each expert, to the chunk's part of slots;
//   before   workgroup e: e's slots in the chunks before each, to their parts of
//            pos, and e's total, to offsets;
//   total    the offsets;
//   scatter  a chunk's places, in slot order: its waves' counts, then lane by
//            lane within groups of 64, whose lanes of one expert find each
//            other bit by bit.  It has read its part of pos before it writes it,
//            and slots is no longer read.
// 262144 slots of 128 experts: 12 us, 45 by sort_kernel, whose every workgroup
// reads every id.
constexpr int64_t kOneLaunch = 65536;
constexpr int kChunk = 2048, kChunkWaves = kChunk / 256;
struct Chunks {  // of `least` slots, the first `more` of one more
  int count, least, more;
  __device__ __forceinline__ int start(int c) const { return c * least + min(c, more); }
};

__global__ void __launch_bounds__(512) sort_count_kernel(const int32_t *ids, Chunks chunks, int n_expert,
                                                         int32_t *slots) {
  __shared__ int counts[QG_MAX_EXPERTS];
  const int i0 = chunks.start((int)blockIdx.x), i1 = chunks.start((int)blockIdx.x + 1);
  for (int e = (int)threadIdx.x; e < n_expert; e += 512) counts[e] = 0;
  __syncthreads();
  for (int i = i0 + (int)threadIdx.x; i < i1; i += 512)
    if ((uint32_t)ids[i] < (uint32_t)n_expert) atomicAdd(&counts[ids[i]], 1);
  __syncthreads();
  for (int e = (int)threadIdx.x; e < n_expert; e += 512) slots[i0 + e] = counts[e];
}

// Inclusive sum over a workgroup of WAVES waves.
template <int WAVES>
__device__ __forceinline__ int scan_add(int v, int *part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  if (lane == 63) part[wave] = v;
  __syncthreads();
  for (int w = 0; w < wave; ++w) v += part[w];
  return v;
}

__global__ void __launch_bounds__(256) sort_before_kernel(const int32_t *slots, Chunks chunks, int32_t *offsets,
                                                          int32_t *pos) {
  __shared__ int part[4];
  const int e = blockIdx.x, per = (chunks.count + 255) / 256;  // each thread's run of chunks
  const int c0 = min((int)threadIdx.x * per, chunks.count), c1 = min(c0 + per, chunks.count);
  int mine = 0;
  for (int c = c0; c < c1; ++c) mine += slots[chunks.start(c) + e];
  const int upto = scan_add<4>(mine, part);
  int at = upto - mine;
  for (int c = c0; c < c1; ++c) {
    const int i = chunks.start(c) + e;
    pos[i] = at;
    at += slots[i];
  }
  if (threadIdx.x == 255) offsets[e + 1] = upto;
}

__global__ void __launch_bounds__(QG_MAX_EXPERTS) sort_total_kernel(int32_t *offsets, int n_expert) {
  __shared__ int part[QG_MAX_EXPERTS / 64];
  const int e = (int)threadIdx.x;
  const int upto = scan_add<QG_MAX_EXPERTS / 64>(e < n_expert ? offsets[e + 1] : 0, part);
  if (e == 0) offsets[0] = 0;
  if (e < n_expert) offsets[e + 1] = upto;
}

__global__ void __launch_bounds__(64 * kChunkWaves) sort_scatter_kernel(const int32_t *ids, Chunks chunks,
                                                                        int n_expert, const int32_t *offsets,
                                                                        int32_t *slots, int32_t *pos) {
  __shared__ int next[kChunkWaves][QG_MAX_EXPERTS];
  constexpr int kThreads = 64 * kChunkWaves;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i0 = chunks.start((int)blockIdx.x), i1 = chunks.start((int)blockIdx.x + 1);
  for (int e = (int)threadIdx.x; e < n_expert; e += kThreads)
#pragma unroll
    for (int w = 0; w < kChunkWaves; ++w) next[w][e] = 0;
  int v[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + 256 * wave + 64 * r + lane;
    v[r] = i < i1 ? ids[i] : -1;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if ((uint32_t)v[r] < (uint32_t)n_expert) atomicAdd(&next[wave][v[r]], 1);
  __syncthreads();
  for (int e = (int)threadIdx.x; e < n_expert; e += kThreads) {
    int at = offsets[e] + pos[i0 + e];
#pragma unroll
    for (int w = 0; w < kChunkWaves; ++w) {
      const int here = next[w][e];
      next[w][e] = at;
      at += here;
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz((uint32_t)n_expert);
  const uint64_t lower = (1ull << lane) - 1;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + 256 * wave + 64 * r + lane, e = v[r];
    const bool kept = (uint32_t)e < (uint32_t)n_expert;
    uint64_t same = __ballot(kept);
    for (int b = 0; b < bits; ++b) {
      const bool one = e >> b & 1;
      const uint64_t ones = __ballot(one);
      same &= one ? ones : ~ones;
    }
    const int rank = __popcll(same & lower);
    if (kept) {
      const int at = next[wave][e] + rank;
      slots[at] = i;
      pos[i] = at;
    } else if (i < i1) {
      pos[i] = -1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (kept && rank == 0) next[wave][e] += __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  const int kept = offsets[n_expert];
  for (int p = max(i0, kept) + (int)threadIdx.x; p < i1; p += kThreads) slots[p] = -1;
}

// `lanes` lanes (a power of two, up to a wave) copy one row at a time, 16 bytes
// each, then the row's last bytes by elements of 2.  Past: more rows than the
// caches hold with what the next kernels read are written past them (32768
// rows of 5760 bytes: 54 us either way, 4.3 TB/s, and the weighted sum of as
// many rows behind it 45 us instead of 62).  Bound by memory; a token's row is
// read once per choice, from the memory side's cache.
template <bool kPast>
__global__ void __launch_bounds__(256) gather_kernel(const uint8_t *x, int64_t x_bytes, int64_t x_rows, int64_t row,
                                                     const int32_t *slots, int n_sel, int64_t n, uint8_t *out,
                                                     int64_t out_bytes, int lanes) {
  const int lane = threadIdx.x & (lanes - 1), per_group = 256 / lanes;
  const int64_t step = (int64_t)gridDim.x * per_group;
  for (int64_t p = (int64_t)blockIdx.x * per_group + threadIdx.x / (unsigned)lanes; p < n; p += step) {
    const int s = slots[p];
    if (s < 0 || s / n_sel >= x_rows) continue;
    const uint8_t *src = x + (int64_t)(s / n_sel) * x_bytes;
    uint8_t *dst = out + p * out_bytes;
    const int64_t whole = row & ~15ll;
    for (int64_t o = 16 * lane; o < whole; o += 16 * lanes) {
      const u32x4 v = *(const u32x4_2 *)(src + o);
      if (kPast) __builtin_nontemporal_store(v, (u32x4_2 *)(dst + o));
      else *(u32x4_2 *)(dst + o) = v;
    }
    for (int64_t o = whole + 2 * lane; o < row; o += 2 * lanes) *(uint16_t *)(dst + o) = *(const uint16_t *)(src + o);
  }
}

// `lanes` lanes (a power of two, up to a wave) take kCols columns of one token
// each; `parts` of them cover its row.  The rows of four choices are loaded
// together, then added one after the other in s order.  8192 tokens of four
// bf16 rows of 2880, written just before: 45 us (5.2 TB/s, as a copy).
constexpr int kCols = 8;
template <int TY, int TO>
__global__ void __launch_bounds__(256) combine_kernel(const uint8_t *y, int64_t y_stride, int64_t y_rows,
                                                      const int32_t *pos, const float *w, int n_sel, int64_t n_cols,
                                                      uint8_t *out, int64_t out_stride, int64_t n_tok, int lanes,
                                                      int parts, int64_t group0) {
  constexpr int EY = Elem<TY>::kSize, EO = Elem<TO>::kSize, kAt = 4;
  const int64_t task = (group0 + blockIdx.x) * (256 / lanes) + threadIdx.x / (unsigned)lanes;
  const int64_t t = parts == 1 ? task : task / parts;
  const int64_t col = ((task - t * parts) * lanes + (threadIdx.x & (lanes - 1))) * kCols;
  if (t >= n_tok || col >= n_cols) return;
  pos += t * n_sel;
  float acc[kCols];
#pragma unroll
  for (int k = 0; k < kCols; ++k) acc[k] = 0.0f;
  const bool whole = col + kCols <= n_cols;
  for (int s0 = 0; s0 < n_sel; s0 += kAt) {
    bool there[kAt];
    float ws[kAt], v[kAt][kCols];
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      const int p = s0 + j < n_sel ? pos[s0 + j] : -1;
      there[j] = p >= 0 && p < y_rows;
      if (!there[j]) continue;
      ws[j] = w ? w[t * n_sel + s0 + j] : 1.0f;
      const uint8_t *src = y + (p * y_stride + col) * EY;
      if (whole) load_n<TY>(src, v[j]);
      else
        for (int k = 0; k < kCols; ++k) {
          float o[1] = {0.0f};
          if (col + k < n_cols) load_n<TY>(src + k * EY, o);
          v[j][k] = o[0];
        }
    }
#pragma unroll
    for (int j = 0; j < kAt; ++j)
      if (there[j])
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] = fmaf(ws[j], v[j][k], acc[k]);
  }
  uint8_t *dst = out + (t * out_stride + col) * EO;
  if (whole) store_n<TO>(dst, acc);
  else
    for (int k = 0; k < kCols; ++k) {
      const float o[1] = {acc[k]};
      if (col + k < n_cols) store_n<TO>(dst + k * EO, o);
    }
}

// A (token, choice) slot's row of dy and its dot product: by a workgroup
// (lanes = 256), or by a power of two of lanes where a row is at most a wave's
// kCols columns each.  The sum goes by lane, then over the lanes, then over the
// waves.  Bound by memory: 4097 x 4 slots of 2880, bf16 rows, fp32 dout: 54 us,
// 4.4 TB/s (6.9 with dout's rows, read once per choice, from the caches).
template <int TD, int TY>
__global__ void __launch_bounds__(256) combine_grad_kernel(const uint8_t *dout, int64_t d_stride, const uint8_t *y,
                                                           int64_t y_stride, int64_t y_rows, const int32_t *pos,
                                                           const float *w, int n_sel, int64_t n_slots, int64_t n_cols,
                                                           uint8_t *dy, int64_t dy_stride, float *dw, int lanes,
                                                           int64_t group0) {
  constexpr int ED = Elem<TD>::kSize, EY = Elem<TY>::kSize;
  __shared__ float part[4];
  const int lane = threadIdx.x & (lanes - 1);
  const int64_t slot = (group0 + blockIdx.x) * (256 / lanes) + threadIdx.x / (unsigned)lanes;
  const int64_t p = slot < n_slots ? pos[slot] : -1;
  const bool there = p >= 0 && p < y_rows;
  float sum = 0.0f;
  if (there) {
    const int64_t t = slot / n_sel;
    const float ws = w[slot];
    const int64_t groups = (n_cols + kCols - 1) / kCols;
    for (int64_t c = lane; c < groups; c += lanes) {
      const int64_t col = kCols * c;
      const uint8_t *d = dout + (t * d_stride + col) * ED;
      const uint8_t *src = y + (p * y_stride + col) * EY;
      uint8_t *dst = dy + (p * dy_stride + col) * EY;
      if (col + kCols <= n_cols) {
        float a[kCols], b[kCols], o[kCols];
        load_n<TD>(d, a);
        load_n<TY>(src, b);
#pragma unroll
        for (int k = 0; k < kCols; ++k) {
          sum = fmaf(a[k], b[k], sum);
          o[k] = ws * a[k];
        }
        store_n<TY>(dst, o);
      } else {
        for (int k = 0; col + k < n_cols; ++k) {
          float a[1], b[1];
          load_n<TD>(d + k * ED, a);
          load_n<TY>(src + k * EY, b);
          sum = fmaf(a[0], b[0], sum);
          const float o[1] = {ws * a[0]};
          store_n<TY>(dst + k * EY, o);
        }
      }
    }
  }
  for (int m = 1; m < min(lanes, 64); m <<= 1) sum += __shfl_xor(sum, m);
  if (lanes == 256) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = (part[0] + part[1]) + (part[2] + part[3]);
  }
  if (lane == 0 && slot < n_slots) dw[slot] = there ? sum : 0.0f;
}

// ---------------------------------------------------------------------------
// Checks
// ---------------------------------------------------------------------------

#define MX_HIP(call)                                                       \
  do {                                                                     \
    hipError_t e_ = (call);                                                \
    if (e_ != hipSuccess) return qgemv_detail::record_hip_error(e_, #call); \
  } while (0)

// f(first, count) for all workgroups of 256 threads, a launch at a time: a
// grid holds fewer than 2^32 threads.
template <typename F>
void in_grids(int64_t groups, F f) {
  constexpr int64_t kMost = 1 << 23;
  for (int64_t first = 0; first < groups; first += kMost) f(first, (unsigned)std::min(groups - first, kMost));
}

constexpr int64_t kMaxDim = 0x7fff0000;  // rows and columns: an index past a tile's end stays an int
constexpr int64_t kMaxStride = 1ll << 40;

int elem_size(int32_t type) { return type == QG_F32 ? 4 : type == QG_F16 || type == QG_BF16 ? 2 : 0; }

// An MXFP4 matrix of at most kMaxDim rows.
int check_mx(const qg_matrix *w) {
  if (!w) return QG_E_NULL;
  if (w->fmt != QG_MXFP4) return QG_E_FMT;
  if (w->k <= 0 || w->k % 32 != 0 || w->k > QG_MAX_K || w->n_rows < 0 || w->n_rows > kMaxDim) return QG_E_SHAPE;
  if (w->reserved != 0) return QG_E_ARG;
  if (w->n_bytes != w->n_rows * (w->k / 32 * 17)) return QG_E_SIZE;
  if (!w->data && w->n_bytes > 0) return QG_E_NULL;
  if ((uintptr_t)w->data & 15) return QG_E_ARG;
  return QG_OK;
}

// blocks: MXFP4 is taken too.  out: rows may not overlap.
int check_tensor(const qg_tensor *t, bool blocks, bool out) {
  if (!t) return QG_E_NULL;
  const int es = elem_size(t->type);
  if (!es && !(blocks && t->type == QG_MXFP4)) return QG_E_FMT;
  if (t->n_rows < 0 || t->n_cols < 0 || t->n_rows > kMaxDim || t->n_cols > kMaxDim) return QG_E_SHAPE;
  if (!es && t->n_cols % 32 != 0) return QG_E_SHAPE;
  if (t->reserved != 0 || t->stride < 0 || t->stride > kMaxStride) return QG_E_ARG;
  if (!es && t->stride != t->n_cols) return QG_E_ARG;
  if (out && t->n_rows > 1 && t->stride < t->n_cols) return QG_E_ARG;
  if (t->n_rows > 0 && t->n_cols > 0 && !t->data) return QG_E_NULL;
  if ((uintptr_t)t->data & (es ? es - 1 : 15)) return QG_E_ARG;
  return QG_OK;
}

int check_window(int64_t n_rows, int64_t r0, int64_t r1) {
  return r0 < 0 || r0 > r1 || r1 > n_rows ? QG_E_RANGE : QG_OK;
}

int launch(int32_t x_type, const MxArgs &a, hipStream_t stream) {
  const auto run = x_type == QG_F32 ? launch_mx<kF32> : x_type == QG_F16 ? launch_mx<kF16>
                   : x_type == QG_BF16 ? launch_mx<kBf16> : launch_mx<kFp4>;
  bool fits = true;
  MX_HIP(run(a, stream, &fits));
  return fits ? QG_OK : QG_E_SHAPE;
}

// Lanes for a row of n pieces: the power of two that covers it, up to a wave.
int row_lanes(int64_t n) {
  int lanes = 1;
  while (lanes < n && lanes < 64) lanes *= 2;
  return lanes;
}

int64_t row_bytes(const qg_tensor *x) {
  return x->type == QG_MXFP4 ? x->n_cols / 32 * 17 : x->stride * elem_size(x->type);
}

int rows_mx(const qg_matrix *w, const qg_matrix *w2, int64_t r0, int64_t r1, const qg_tensor *x, const qg_tensor *y,
            hipStream_t stream) {
  int rc;
  if ((rc = check_mx(w)) || (w2 && (rc = check_mx(w2)))) return rc;
  if (w2 && (w2->n_rows != w->n_rows || w2->k != w->k)) return QG_E_SHAPE;
  if ((rc = check_window(w->n_rows, r0, r1)) || (rc = check_tensor(x, true, false)) ||
      (rc = check_tensor(y, false, true)))
    return rc;
  if (x->n_cols != w->k || y->n_rows != x->n_rows || y->n_cols != r1 - r0) return QG_E_SHAPE;
  if (x->n_rows == 0 || r0 == r1) return QG_OK;
  MxArgs a = {};
  const int64_t rb = w->k / 32 * 17;
  a.w = (const uint8_t *)w->data + r0 * rb;
  a.w2 = w2 ? (const uint8_t *)w2->data + r0 * rb : nullptr;
  a.x = (const uint8_t *)x->data;
  a.y = y->data;
  a.x_bytes = row_bytes(x);
  a.y_stride = y->stride;
  a.row_bytes = (int32_t)rb;
  a.nb = (int32_t)(w->k / 32);
  a.n = (int32_t)(r1 - r0);
  a.places = (int32_t)x->n_rows;
  a.x_rows = (int32_t)x->n_rows;
  a.n_expert = a.n_sel = 1;
  a.y_type = y->type;
  return launch(x->type, a, stream);
}

int expert_mx(const qg_matrix *w, const qg_matrix *w2, int64_t n_expert, const qg_tensor *x, const int32_t *offsets,
              const int32_t *slots, int32_t n_sel, const qg_tensor *y, hipStream_t stream) {
  int rc;
  if ((rc = check_mx(w)) || (w2 && (rc = check_mx(w2)))) return rc;
  if (w2 && (w2->n_rows != w->n_rows || w2->k != w->k)) return QG_E_SHAPE;
  if ((rc = check_tensor(x, true, false)) || (rc = check_tensor(y, false, true))) return rc;
  if (n_expert < 1 || n_expert > QG_MAX_EXPERTS || w->n_rows % n_expert != 0) return QG_E_SHAPE;
  const int64_t out = w->n_rows / n_expert;
  if (x->n_cols != w->k || y->n_cols != out || (!slots && x->n_rows < y->n_rows)) return QG_E_SHAPE;
  if (slots && n_sel < 1) return QG_E_ARG;
  if (y->n_rows == 0 || out == 0) return QG_OK;
  if (!offsets) return QG_E_NULL;
  MxArgs a = {};
  a.w = (const uint8_t *)w->data;
  a.w2 = w2 ? (const uint8_t *)w2->data : nullptr;
  a.x = (const uint8_t *)x->data;
  a.y = y->data;
  a.offsets = offsets;
  a.slots = slots;
  a.row_bytes = (int32_t)(w->k / 32 * 17);
  a.expert_bytes = out * a.row_bytes;
  a.x_bytes = row_bytes(x);
  a.y_stride = y->stride;
  a.nb = x->n_rows > 0 ? (int32_t)(w->k / 32) : 0;  // without any row of x every sum is empty
  a.n = (int32_t)out;
  a.places = (int32_t)y->n_rows;
  a.x_rows = (int32_t)x->n_rows;
  a.n_expert = (int32_t)n_expert;
  a.n_sel = slots ? n_sel : 1;
  a.y_type = y->type;
  return launch(x->type, a, stream);
}

// f(integral_constant<type>) for a checked float type.
template <typename F>
void with_type(int32_t type, F f) {
  if (type == QG_F32) f(std::integral_constant<int, QG_F32>());
  else if (type == QG_F16) f(std::integral_constant<int, QG_F16>());
  else f(std::integral_constant<int, QG_BF16>());
}

}  // namespace

extern "C" {

int qgemv_mx_quantize(const qg_tensor *x, const qg_matrix *q, qg_stream_t stream) {
  int rc;
  if ((rc = check_mx(q)) || (rc = check_tensor(x, false, false))) return rc;
  if (x->n_rows != q->n_rows || x->n_cols != q->k) return QG_E_SHAPE;
  if (x->n_rows == 0) return QG_OK;
  const int nb = (int)(q->k / 32);
  const int64_t blocks = q->n_rows * nb, grid = (blocks + kQBlocks - 1) / kQBlocks;
  with_type(x->type, [&](auto T) {
    in_grids(grid, [&](int64_t first, unsigned count) {
      hipLaunchKernelGGL(quantize_kernel<decltype(T)::value>, dim3(count), dim3(256), 0, stream,
                         (const uint8_t *)x->data, x->stride, nb, blocks, (uint8_t *)q->data, first);
    });
  });
  MX_HIP(hipGetLastError());
  return QG_OK;
}

int qgemv_mx_dequantize(const qg_matrix *q, int64_t row_start, int64_t row_end, const qg_tensor *out,
                        qg_stream_t stream) {
  int rc;
  if ((rc = check_mx(q)) || (rc = check_window(q->n_rows, row_start, row_end)) ||
      (rc = check_tensor(out, false, true)))
    return rc;
  if (out->n_rows != row_end - row_start || out->n_cols != q->k) return QG_E_SHAPE;
  if (out->n_rows == 0) return QG_OK;
  const int nb = (int)(q->k / 32);
  const int64_t blocks = out->n_rows * nb, grid = (blocks + 63) / 64;
  with_type(out->type, [&](auto T) {
    in_grids(grid, [&](int64_t first, unsigned count) {
      hipLaunchKernelGGL(dequantize_kernel<decltype(T)::value>, dim3(count), dim3(256), 0, stream,
                         (const uint8_t *)q->data + row_start * nb * 17, nb, blocks, (uint8_t *)out->data, out->stride,
                         first);
    });
  });
  MX_HIP(hipGetLastError());
  return QG_OK;
}

int qgemv_rows_mx(const qg_matrix *w, int64_t row_start, int64_t row_end, const qg_tensor *x, const qg_tensor *y,
                  qg_stream_t stream) {
  return rows_mx(w, nullptr, row_start, row_end, x, y, stream);
}

int qgemv_rows_mx_swiglu(const qg_matrix *gate, const qg_matrix *up, int64_t row_start, int64_t row_end,
                         const qg_tensor *x, const qg_tensor *h, qg_stream_t stream) {
  if (!gate || !up) return QG_E_NULL;
  return rows_mx(gate, up, row_start, row_end, x, h, stream);
}

int qgemv_expert_mx(const qg_matrix *w, int64_t n_expert, const qg_tensor *x, const int32_t *offsets,
                    const int32_t *slots, int32_t n_sel, const qg_tensor *y, qg_stream_t stream) {
  return expert_mx(w, nullptr, n_expert, x, offsets, slots, n_sel, y, stream);
}

int qgemv_expert_mx_swiglu(const qg_matrix *gate, const qg_matrix *up, int64_t n_expert, const qg_tensor *x,
                           const int32_t *offsets, const int32_t *slots, int32_t n_sel, const qg_tensor *h,
                           qg_stream_t stream) {
  if (!gate || !up) return QG_E_NULL;
  return expert_mx(gate, up, n_expert, x, offsets, slots, n_sel, h, stream);
}

int qgemv_expert_sort(const int32_t *ids, int64_t n_tok, int32_t n_sel, int64_t n_expert, int32_t *offsets,
                      int32_t *slots, int32_t *pos, qg_stream_t stream) {
  if (n_tok < 0 || n_sel < 1) return QG_E_ARG;
  if (n_expert < 1 || n_expert > QG_MAX_EXPERTS || n_tok > (1ll << 30) / n_sel) return QG_E_SHAPE;
  const int64_t n = n_tok * n_sel;
  if (!offsets || (n > 0 && (!ids || !slots || !pos))) return QG_E_NULL;
  // One launch's workgroups read every id each, a round of 256 experts at a
  // time (65536 slots of 128 experts 15 us, of 1024 38; 16384 of 1024 about 14);
  // four launches take 10 to 13 up to a million slots, and more of the host.
  if (n * ((n_expert + 255) / 256) <= kOneLaunch) {
    hipLaunchKernelGGL(sort_kernel, dim3((unsigned)n_expert + 1), dim3(64 * kSortWaves), 0, stream, ids, (int)n,
                       (int)n_expert, offsets, slots, pos);
  } else {
    const int count = (int)((n + kChunk - 1) / kChunk);
    const Chunks chunks = {count, (int)n / count, (int)n % count};
    constexpr int64_t kLeast = kOneLaunch / ((QG_MAX_EXPERTS + 255) / 256) + 1;
    static_assert(kLeast / ((kLeast + kChunk - 1) / kChunk) >= QG_MAX_EXPERTS, "a chunk holds its table");
    hipLaunchKernelGGL(sort_count_kernel, dim3(chunks.count), dim3(512), 0, stream, ids, chunks, (int)n_expert, slots);
    hipLaunchKernelGGL(sort_before_kernel, dim3((unsigned)n_expert), dim3(256), 0, stream, slots, chunks, offsets, pos);
    hipLaunchKernelGGL(sort_total_kernel, dim3(1), dim3(QG_MAX_EXPERTS), 0, stream, offsets, (int)n_expert);
    hipLaunchKernelGGL(sort_scatter_kernel, dim3(chunks.count), dim3(64 * kChunkWaves), 0, stream, ids, chunks,
                       (int)n_expert, offsets, slots, pos);
  }
  MX_HIP(hipGetLastError());
  return QG_OK;
}

int qgemv_expert_gather(const qg_tensor *x, const int32_t *slots, int32_t n_sel, const qg_tensor *out,
                        qg_stream_t stream) {
  int rc;
  if ((rc = check_tensor(x, false, false)) || (rc = check_tensor(out, false, true))) return rc;
  if (x->type != out->type) return QG_E_FMT;
  if (x->n_cols != out->n_cols) return QG_E_SHAPE;
  if (n_sel < 1) return QG_E_ARG;
  if (out->n_rows == 0 || out->n_cols == 0) return QG_OK;
  if (!slots) return QG_E_NULL;
  const int es = elem_size(x->type);
  const int lanes = row_lanes((out->n_cols * es + 15) / 16);
  const unsigned grid = (unsigned)std::min<int64_t>((out->n_rows * lanes + 255) / 256, 1 << 20);
  // (the memory-side cache holds 256 MB)
  const auto kernel = out->n_rows * out->n_cols * es > (64ll << 20) ? gather_kernel<true> : gather_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, stream, (const uint8_t *)x->data, x->stride * es, x->n_rows,
                     x->n_cols * es, slots, n_sel, out->n_rows, (uint8_t *)out->data, out->stride * es, lanes);
  MX_HIP(hipGetLastError());
  return QG_OK;
}

int qgemv_expert_combine(const qg_tensor *y, const int32_t *pos, const float *w, int32_t n_sel, const qg_tensor *out,
                         qg_stream_t stream) {
  int rc;
  if ((rc = check_tensor(y, false, false)) || (rc = check_tensor(out, false, true))) return rc;
  if (y->n_cols != out->n_cols) return QG_E_SHAPE;
  if (n_sel < 0) return QG_E_ARG;
  if (n_sel > 1 << 30) return QG_E_SHAPE;
  if (out->n_rows == 0 || out->n_cols == 0) return QG_OK;
  if (n_sel > 0 && !pos) return QG_E_NULL;
  const int lanes = row_lanes((out->n_cols + kCols - 1) / kCols);
  const int64_t parts = (out->n_cols + lanes * kCols - 1) / (lanes * kCols);
  const int64_t grid = (out->n_rows * parts * lanes + 255) / 256;
  with_type(y->type, [&](auto TY) {
    with_type(out->type, [&](auto TO) {
      in_grids(grid, [&](int64_t first, unsigned count) {
        hipLaunchKernelGGL((combine_kernel<decltype(TY)::value, decltype(TO)::value>), dim3(count), dim3(256), 0,
                           stream, (const uint8_t *)y->data, y->stride, y->n_rows, pos, w, (int)n_sel, out->n_cols,
                           (uint8_t *)out->data, out->stride, out->n_rows, lanes, (int)parts, first);
      });
    });
  });
  MX_HIP(hipGetLastError());
  return QG_OK;
}

int qgemv_expert_combine_grad(const qg_tensor *dout, const qg_tensor *y, const int32_t *pos, const float *w,
                              int32_t n_sel, const qg_tensor *dy, float *dw, qg_stream_t stream) {
  int rc;
  if ((rc = check_tensor(dout, false, false)) || (rc = check_tensor(y, false, false)) ||
      (rc = check_tensor(dy, false, true)))
    return rc;
  if (dy->type != y->type) return QG_E_FMT;
  if (dout->n_cols != y->n_cols || dy->n_cols != y->n_cols || dy->n_rows != y->n_rows) return QG_E_SHAPE;
  if (n_sel < 1) return QG_E_ARG;
  if (dout->n_rows > (1ll << 30) / n_sel) return QG_E_SHAPE;
  if (y->n_rows > 0 && y->data == dy->data && y->n_cols > 0) return QG_E_ARG;
  if (dout->n_rows == 0) return QG_OK;
  if (!pos || !w || !dw) return QG_E_NULL;
  const int64_t groups = (y->n_cols + kCols - 1) / kCols, slots = dout->n_rows * n_sel;
  const int lanes = groups > 64 ? 256 : row_lanes(groups);
  with_type(dout->type, [&](auto TD) {
    with_type(y->type, [&](auto TY) {
      in_grids((slots * lanes + 255) / 256, [&](int64_t first, unsigned count) {
        hipLaunchKernelGGL((combine_grad_kernel<decltype(TD)::value, decltype(TY)::value>), dim3(count), dim3(256), 0,
                           stream, (const uint8_t *)dout->data, dout->stride, (const uint8_t *)y->data, y->stride,
                           y->n_rows, pos, w, (int)n_sel, slots, dout->n_cols, (uint8_t *)dy->data, dy->stride, dw,
                           lanes, first);
      });
    });
  });
  MX_HIP(hipGetLastError());
  return QG_OK;
}

}  // extern "C"
