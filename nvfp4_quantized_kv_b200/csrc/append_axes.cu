// append_axes.cu -- nvkv_append_rope_axes: rotary positions with several
// axes (time, height, width, ...) for the new K rows and queries, fused with
// the quantised write of K and V into the NVFP4 paged pool: one launch reads
// every new row once.
//
// Pair i (elements i and i + rotary_dim/2) of every head of row r turns by
// table row positions[axis_of_pair[i]][r]:
//     x' = fma(x, c, -(y*s)),  y' = fma(y, c, x*s)      (products rounded)
// K is then quantised as by nvkv_append_rope, the queries are rounded to bf16.
//
// Bound by HBM for long chunks and by the latency of its dependent loads
// (lengths, page id, row) for single rows.  Two kinds of warps:
//  * row warps take 8 heads of one row (K heads or query heads).  D/16 lanes
//    hold a head, 16 elements each: a rotated lane the 8 elements 8l.. and
//    their partners, so the pairs' cosines are loaded once for all heads of
//    the warp and no element is loaded twice; a group of 16 is then two
//    neighbouring lanes.  Lanes past rotary_dim hold one whole group.  Eight
//    heads a warp leave a batch of single rows enough warps (4 a row at 24/4
//    heads) and read the row's table 4 times, from L2.
//  * V warps take half a page (8 slots) of one kv-head (of two at head_dim
//    128), 8 head_dim elements a lane, and gather the nibbles of the new slots
//    in registers: V is stored transposed, so 8 new slots leave as one word
//    an element; otherwise only the bytes of slot pairs with a new slot are
//    written (the other nibble of such a byte is kept).  They come first in
//    the grid and load their 8 rows at once: one warp for a whole page, row
//    after row, at the grid's end, made the launch twice as long.
//
// Measured (24/4 heads, head_dim 256, queries included): 2,048 rows, rotary
// width 128: 15.2 us, 61 MB = 4,020 GB/s, 0.61 of the measured copy rate (4
// blocks an SM are one wave and a half of dependent loads); one row for each
// of 64 sequences: 6.6 us, the launch and four dependent loads.
#include "nvkv_common.cuh"

namespace nvkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeadsPerWarp = 8;
constexpr int kMaxAxes = 4;

struct AxisMap {
  alignas(8) uint8_t axis[128];  // of each pair
};

__device__ __forceinline__ void unpack8(const uint4 &r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Asynchronous 16-byte copy into the thread's own slot of shared memory.  The
// new rows wait there instead of in registers, so twice as many warps fit
// and twice as many rows are on their way.
__device__ __forceinline__ void fetch16(uint4 *slot, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(slot)),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void fetched() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// One pair turned, in the stated order of roundings.
__device__ __forceinline__ void turn_pair(float &x, float &y, float c, float s) {
  const float ys = __fmul_rn(y, s), xs = __fmul_rn(x, s);
  x = fmaf(x, c, -ys);
  y = fmaf(y, c, xs);
}

// Two pairs of bf16 elements (one word each side), rounded back to bf16.
__device__ __forceinline__ void turn_words(uint32_t &xw, uint32_t &yw, const float *c,
                                           const float *s) {
  float x0 = __uint_as_float(xw << 16), x1 = __uint_as_float(xw & 0xffff0000u);
  float y0 = __uint_as_float(yw << 16), y1 = __uint_as_float(yw & 0xffff0000u);
  turn_pair(x0, y0, c[0], s[0]);
  turn_pair(x1, y1, c[1], s[1]);
  const __nv_bfloat162 xr = __floats2bfloat162_rn(x0, x1), yr = __floats2bfloat162_rn(y0, y1);
  xw = *reinterpret_cast<const uint32_t *>(&xr);
  yw = *reinterpret_cast<const uint32_t *>(&yr);
}

// The largest |x| of 8 values as float bits; infinities and NaN compare
// above every number.
__device__ __forceinline__ uint32_t amax8(const float (&x)[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(x[i]) & 0x7fffffffu);
  return a;
}

constexpr uint32_t kInfBits = 0x7f800000u;

// The largest number among 8 values (NaN left out), as nvkv_append takes it.
__device__ __noinline__ float amax8_numbers(const float (&x)[8]) {
  float a = 0.f;
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
  return a;
}

__device__ __noinline__ uint32_t codes8_compare(const float (&x)[8], float s) {
  uint32_t c = 0;
  for (int i = 0; i < 8; ++i) c |= e2m1_code(x[i], s) << (4 * i);
  return c;
}

// The codes of 8 elements under a scale byte (element 0 in bits 0..3): the
// hardware's round-to-nearest-even conversion of x / s.  It decides like the
// exact comparison of |x| with every midpoint m * s because the quotient is
// correctly rounded and rounding keeps order: the quotient is m only when x
// is m * s (their next floats are more than half a step of m away, s having
// 4 significant bits).  Correctly rounded division with the rounded
// reciprocal r of s and one residual, x r + (x - x r s) r, is Markstein's;
// 3 instructions an element where the comparisons take 14.  Values
// that are not finite take the comparisons (`plain` false).
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], uint32_t scale, bool plain) {
  if (scale == 0) return 0u;
  const float s = e4m3_to_float((uint8_t)scale);
  if (!plain) return codes8_compare(x, s);
  const float r = __frcp_rn(s);
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float q0 = x[2 * i] * r, q1 = x[2 * i + 1] * r;
    q0 = fmaf(fmaf(-q0, s, x[2 * i]), r, q0);
    q1 = fmaf(fmaf(-q1, s, x[2 * i + 1]), r, q1);
    c |= f32x2_to_e2m1x2(q0, q1) << (8 * i);
  }
  // a magnitude that rounds to 0 is code 0, without its sign
  const uint32_t some = (c | (c >> 1) | (c >> 2)) & 0x11111111u;
  return c & (0x77777777u | (some << 3));
}

// Scale byte of a group whose largest |x| has the bits a.
__device__ __forceinline__ uint32_t scale_of(uint32_t a) {
  return scale_byte_of_amax(__uint_as_float(a));
}

// 8 words of 8 nibbles, transposed: nibble j of word i <-> nibble i of word j.
__device__ __forceinline__ void transpose_nibbles(uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 16-bit halves, words i and i + 4
    const uint32_t a = w[i], b = w[i + 4];
    w[i] = __byte_perm(a, b, 0x5410);
    w[i + 4] = __byte_perm(a, b, 0x7632);
  }
#pragma unroll
  for (int g = 0; g < 8; g += 4)
#pragma unroll
    for (int i = g; i < g + 2; ++i) {  // bytes, words i and i + 2
      const uint32_t a = w[i], b = w[i + 2];
      w[i] = __byte_perm(a, b, 0x6240);
      w[i + 2] = __byte_perm(a, b, 0x7351);
    }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {  // nibbles, words i and i + 1
    const uint32_t a = w[i], b = w[i + 1];
    w[i] = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
    w[i + 1] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
  }
}

// The positions of row `row` on every axis, all loads at once; whether each
// has a table row.
__device__ __forceinline__ bool positions_of(const int32_t *pos, int axes, int total, int row,
                                             int max_pos, int (&p)[kMaxAxes]) {
#pragma unroll
  for (int a = 0; a < kMaxAxes; ++a) p[a] = a < axes ? pos[(size_t)a * total + row] : 0;
  bool ok = true;
#pragma unroll
  for (int a = 0; a < kMaxAxes; ++a) ok &= p[a] >= 0 && p[a] < max_pos;
  return ok;
}

__device__ __forceinline__ float4 load_two(const float *a, const float *b) {
  const float2 x = __ldg(reinterpret_cast<const float2 *>(a));
  const float2 y = __ldg(reinterpret_cast<const float2 *>(b));
  return make_float4(x.x, x.y, y.x, y.y);
}

struct Args {
  uint8_t *pool;
  int num_pages, Hkv;
  const int32_t *page_table;
  int max_pages;
  const int32_t *kv_lens;
  int max_kv_len;
  const __nv_bfloat16 *k, *v, *q;  // q null: no queries
  __nv_bfloat16 *q_out;
  int Hq;
  const int32_t *cu_new;
  int total_new, max_new;
  const float *cs;  // 8-byte aligned; cs16: 16-byte
  bool cs16;
  int max_pos, rotary_dim;
  const int32_t *positions;
  int axes;
  int32_t *err;
};

template <int D>
__device__ __forceinline__ void append_v(const Args &a, int b, int wid, int row0, int first,
                                         int len, uint4 *stage) {
  const int lane = threadIdx.x & 31;
  constexpr int lanes = D / 8;
  const int l = lane % lanes;
  const int64_t ph = (int64_t)(wid >> 1) * (32 / lanes) + lane / lanes;
  const int half = wid & 1;  // slots 8 * half .. 8 * half + 7
  const int h = (int)(ph % a.Hkv);
  const int64_t pi = first / kPageTokens + ph / a.Hkv;
  bool live = pi * kPageTokens < len;
  const int p0 = live ? (int)pi * kPageTokens + 8 * half : 0;  // position of the first slot
  // Everything the unit needs is asked for before anything is waited for.
  const __nv_bfloat16 *src =
      a.v + ((int64_t)row0 + p0 - first) * (int64_t)a.Hkv * D + (size_t)h * D + 8 * l;
#pragma unroll
  for (int sl = 0; sl < 8; ++sl)
    if (live && p0 + sl >= first && p0 + sl < len)
      fetch16(stage + 32 * sl, src + (int64_t)sl * a.Hkv * D);
  int page = -1;
  if (live) page = a.page_table[(size_t)b * a.max_pages + pi];
  bool ok = false;
  {
    const int pos = p0 + (lane & 7);
    int p[kMaxAxes];
    if (live && pos >= first && pos < len)
      ok = positions_of(a.positions, a.axes, a.total_new, row0 + pos - first, a.max_pos, p);
  }
  live = page >= 0 && page < a.num_pages;  // (a bad one is reported by the row warps)
  // New slots: inside [first, len), with a table row.  (At head_dim 128 each
  // half-warp votes on a page of its own.)
  const uint32_t fresh = (__ballot_sync(0xffffffffu, ok && live) >> (lane & 16)) & 0xffu;
  fetched();
  if (!__any_sync(0xffffffffu, fresh != 0)) return;
  uint32_t w[8];              // slot s: the codes of the 8 elements
  uint32_t sc[2] = {0u, 0u};  // the slots' scale bytes
#pragma unroll
  for (int sl = 0; sl < 8; ++sl) {
    float x[8];
    unpack8((fresh >> sl) & 1u ? stage[32 * sl] : make_uint4(0u, 0u, 0u, 0u), x);
    uint32_t ax = amax8(x);
    ax = max(ax, __shfl_xor_sync(0xffffffffu, ax, 1));
    const bool plain = ax < kInfBits;
    if (__any_sync(0xffffffffu, !plain)) {  // rare
      float m = amax8_numbers(x);
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      ax = __float_as_uint(m);
    }
    const uint32_t sb = scale_of(ax);
    w[sl] = codes8(x, sb, plain);
    sc[sl >> 2] |= sb << (8 * (sl & 3));
  }
  transpose_nibbles(w);  // element e: the codes of the 8 slots
  if (fresh == 0) return;
  uint8_t *blk = a.pool + ((size_t)page * a.Hkv + h) * head_bytes(D);
  uint8_t *vc = blk + vc_off(D) + 64 * l + 4 * half;
  uint8_t *vs = blk + vs_off(D) + (l >> 1) * kPageTokens + 8 * half;
  if (fresh == 0xffu) {
#pragma unroll
    for (int e = 0; e < 8; ++e) *reinterpret_cast<uint32_t *>(vc + 8 * e) = w[e];
    if ((l & 1) == 0) *reinterpret_cast<uint2 *>(vs) = make_uint2(sc[0], sc[1]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // slot pair (2j, 2j + 1): byte j of each element
    const uint32_t two = (fresh >> (2 * j)) & 3u;
    if (two == 0) continue;
    const uint32_t keep = two == 3u ? 0u : two == 1u ? 0xf0u : 0x0fu;
    uint32_t old[8] = {};
    if (keep) {
#pragma unroll
      for (int e = 0; e < 8; ++e) old[e] = vc[8 * e + j] & keep;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) vc[8 * e + j] = (uint8_t)(((w[e] >> (8 * j)) & ~keep) | old[e]);
    if ((l & 1) == 0) {
      if (two & 1u) vs[2 * j] = (uint8_t)(sc[j >> 1] >> (16 * (j & 1)));
      if (two & 2u) vs[2 * j + 1] = (uint8_t)(sc[j >> 1] >> (16 * (j & 1) + 8));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 4)
append_axes_kernel(const Args a, const __grid_constant__ AxisMap map, int v_warps) {
  const int b = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int wid = blockIdx.x * kWarps + (threadIdx.x >> 5);
  __shared__ uint4 s_stage[kWarps][8 * 32];
  uint4 *stage = s_stage[threadIdx.x >> 5] + lane;  // this thread's slots: every 32nd

  const int row0 = a.cu_new[b], n = a.cu_new[b + 1] - row0, len = a.kv_lens[b];
  if (n <= 0) return;
  const int first = len - n;  // position of the first new row
  if (row0 < 0 || row0 > a.total_new - n || n > a.max_new || first < 0 || len > a.max_kv_len ||
      len > a.max_pages * kPageTokens) {
    if (wid == 0 && lane == 0) report(a.err, NVKV_DEVERR_LENGTH);
    return;
  }
  const int32_t *pt = a.page_table + (size_t)b * a.max_pages;
  auto page_at = [&](int pos) -> int {
    const int p = pt[pos / kPageTokens];
    return p >= 0 && p < a.num_pages ? p : -1;
  };

  // The V warps come first: theirs is the longer chain.
  if (wid < v_warps) {
    append_v<D>(a, b, wid, row0, first, len, stage);
    return;
  }
  {
    // ---------------------------------------------- K heads or query heads
    const int kchunks = (a.Hkv + kHeadsPerWarp - 1) / kHeadsPerWarp;
    const int qchunks = a.q ? (a.Hq + kHeadsPerWarp - 1) / kHeadsPerWarp : 0;
    const int i = (wid - v_warps) / (kchunks + qchunks);
    const int chunk = (wid - v_warps) % (kchunks + qchunks);
    if (i >= n) return;
    const int row = row0 + i, pos = first + i;
    const bool is_q = chunk >= kchunks;
    constexpr int lanes = D / 16;                // of a head
    constexpr int kPasses = kHeadsPerWarp * lanes / 32;
    const int l = lane % lanes, sub = lane / lanes;
    const int half = a.rotary_dim / 2;
    const bool turn = 8 * l < half;
    // elements of this lane: [e0, e0 + 8) and [e1, e1 + 8)
    const int e0 = turn ? 8 * l : a.rotary_dim + 16 * (l - half / 8);
    const int e1 = turn ? half + 8 * l : e0 + 8;
    // Everything the warp needs is asked for before anything is waited for:
    // its heads, the page id, the positions and then their table rows.
    const int heads = is_q ? a.Hq : a.Hkv;
    const int h0 = (is_q ? chunk - kchunks : chunk) * kHeadsPerWarp;
    const __nv_bfloat16 *src = (is_q ? a.q : a.k) + ((size_t)row * heads + h0 + sub) * D;
#pragma unroll
    for (int i2 = 0; i2 < kPasses; ++i2) {
      if (h0 + i2 * (32 / lanes) + sub < heads) {
        const __nv_bfloat16 *hs = src + (size_t)i2 * (32 / lanes) * D;
        fetch16(stage + 64 * i2, hs + e0);
        fetch16(stage + 64 * i2 + 32, hs + e1);
      }
    }
    uint2 axis8 = make_uint2(0u, 0u);  // the axes of the lane's 8 pairs
    if (turn) axis8 = *reinterpret_cast<const uint2 *>(map.axis + 8 * l);
    int p[kMaxAxes];
    const bool in_table = positions_of(a.positions, a.axes, a.total_new, row, a.max_pos, p);
    const int page = page_at(pos);
    if (page < 0) {
      if (chunk == 0 && lane == 0) report(a.err, NVKV_DEVERR_PAGE_ID);
      if (!is_q) return;
    }
    if (!in_table) {
      if (chunk == 0 && lane == 0) report(a.err, NVKV_DEVERR_LENGTH);
      return;
    }
    float c[8], sn[8];  // of the lane's 8 pairs
    {
      auto at = [&](int e) {  // the position that pair e turns by
        const uint32_t ax = ((e < 4 ? axis8.x : axis8.y) >> (8 * (e & 3))) & 3u;
        return ax < 2 ? (ax ? p[1] : p[0]) : (ax == 2 ? p[2] : p[3]);
      };
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // two pairs; mostly of one axis
        float4 v = make_float4(1.f, 0.f, 1.f, 0.f);
        if (turn) {
          const int a0 = at(2 * e), a1 = at(2 * e + 1);
          const float *cs0 = a.cs + (size_t)a0 * a.rotary_dim + 16 * l + 4 * e;
          if (a0 == a1) {
            v = a.cs16 ? __ldg(reinterpret_cast<const float4 *>(cs0)) : load_two(cs0, cs0 + 2);
          } else {
            v = load_two(cs0, a.cs + (size_t)a1 * a.rotary_dim + 16 * l + 4 * e + 2);
          }
        }
        c[2 * e] = v.x, c[2 * e + 1] = v.z;
        sn[2 * e] = v.y, sn[2 * e + 1] = v.w;
      }
    }
    fetched();
    if (is_q) {
      __nv_bfloat16 *dst = a.q_out + ((size_t)row * heads + h0 + sub) * D;
#pragma unroll
      for (int i2 = 0; i2 < kPasses; ++i2) {
        if (h0 + i2 * (32 / lanes) + sub >= heads) break;
        uint4 xw = stage[64 * i2], yw = stage[64 * i2 + 32];
        if (turn) {
          turn_words(xw.x, yw.x, c + 0, sn + 0);
          turn_words(xw.y, yw.y, c + 2, sn + 2);
          turn_words(xw.z, yw.z, c + 4, sn + 4);
          turn_words(xw.w, yw.w, c + 6, sn + 6);
        }
        *reinterpret_cast<uint4 *>(dst + (size_t)i2 * (32 / lanes) * D + e0) = xw;
        *reinterpret_cast<uint4 *>(dst + (size_t)i2 * (32 / lanes) * D + e1) = yw;
      }
      return;
    }
#pragma unroll
    for (int i2 = 0; i2 < kPasses; ++i2) {
      const int h = h0 + i2 * (32 / lanes) + sub;
      const bool live = h < heads;
      if (h0 + i2 * (32 / lanes) >= heads) break;  // warp-uniform
      float x[8], y[8];
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      unpack8(live ? stage[64 * i2] : zero, x);
      unpack8(live ? stage[64 * i2 + 32] : zero, y);
      if (turn) {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn_pair(x[e], y[e], c[e], sn[e]);
      }
      // group maxima: a rotated group is this lane and its neighbour
      uint32_t ax = amax8(x), ay = amax8(y);
      const bool plain = max(ax, ay) < kInfBits;
      if (__any_sync(0xffffffffu, !plain)) {  // rare
        ax = __float_as_uint(amax8_numbers(x));
        ay = __float_as_uint(amax8_numbers(y));
      }
      const uint32_t nx = __shfl_xor_sync(0xffffffffu, ax, 1), ny = __shfl_xor_sync(0xffffffffu, ay, 1);
      ax = turn ? max(ax, nx) : max(ax, ay);
      ay = turn ? max(ay, ny) : ax;
      const uint32_t sx = scale_of(ax), sy = scale_of(ay);
      const uint32_t cx = codes8(x, sx, plain), cy = codes8(y, sy, plain);
      if (!live) continue;
      const int slot = pos % kPageTokens;
      uint8_t *blk = a.pool + ((size_t)page * a.Hkv + h) * head_bytes(D);
      *reinterpret_cast<uint32_t *>(blk + kc_off(D) + slot * (D / 2) + e0 / 2) = cx;
      *reinterpret_cast<uint32_t *>(blk + kc_off(D) + slot * (D / 2) + e1 / 2) = cy;
      uint8_t *ks = blk + ks_off(D) + slot * (D / 16);
      if (turn) {
        // even lane: the x group's scale, odd lane: the y group's
        if (l & 1)
          ks[e1 / 16] = (uint8_t)sy;
        else
          ks[e0 / 16] = (uint8_t)sx;
      } else {
        ks[e0 / 16] = (uint8_t)sx;
      }
    }
  }
}

}  // namespace

// Warps of one sequence's share of the grid.
static int64_t row_warps_of(const nvkv_cache &c, int max_new, int Hq, bool has_q) {
  const int chunks = (c.num_kv_heads + kHeadsPerWarp - 1) / kHeadsPerWarp +
                     (has_q ? (Hq + kHeadsPerWarp - 1) / kHeadsPerWarp : 0);
  return (int64_t)max_new * chunks;
}
static int64_t v_warps_of(const nvkv_cache &c, int max_new) {
  const int64_t pages = ((int64_t)max_new + 2 * kPageTokens - 2) / kPageTokens;
  const int per_warp = 256 / c.head_dim;
  return (pages * c.num_kv_heads + per_warp - 1) / per_warp * 2;
}

// Whether the kernel's 32-bit warp index holds the call.
bool append_axes_fits(const nvkv_cache &c, int max_new, int Hq, bool has_q) {
  return row_warps_of(c, max_new, Hq, has_q) + v_warps_of(c, max_new) + kWarps <= INT32_MAX;
}

int append_axes_max_axes() { return kMaxAxes; }

cudaError_t launch_append_axes(const nvkv_cache &c, const nvkv_seqs &s, const void *k_new,
                               const void *v_new, const int32_t *cu_new, int total_new,
                               int max_new, const float *cs, int max_pos, int rotary_dim,
                               const int32_t *positions, int axes, const uint8_t *axis_of_pair,
                               const void *q, int Hq, void *q_out, cudaStream_t stream) {
  Args a;
  a.pool = c.pool, a.num_pages = c.num_pages, a.Hkv = c.num_kv_heads;
  a.page_table = s.page_table, a.max_pages = s.max_pages_per_seq;
  a.kv_lens = s.kv_lens, a.max_kv_len = s.max_kv_len;
  a.k = static_cast<const __nv_bfloat16 *>(k_new);
  a.v = static_cast<const __nv_bfloat16 *>(v_new);
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.q_out = static_cast<__nv_bfloat16 *>(q_out);
  a.Hq = Hq, a.cu_new = cu_new, a.total_new = total_new, a.max_new = max_new;
  a.cs16 = (reinterpret_cast<uintptr_t>(cs) & 15u) == 0;
  a.cs = cs, a.max_pos = max_pos, a.rotary_dim = rotary_dim;
  a.positions = positions, a.axes = axes, a.err = s.err_word;
  AxisMap map{};
  for (int i = 0; i < rotary_dim / 2; ++i) map.axis[i] = axis_of_pair[i];
  const int v_warps = (int)v_warps_of(c, max_new);
  const int64_t warps = v_warps + row_warps_of(c, max_new, Hq, q != nullptr);
  const dim3 grid((unsigned)((warps + kWarps - 1) / kWarps), (unsigned)s.batch);
  auto kernel = c.head_dim == 256 ? append_axes_kernel<256> : append_axes_kernel<128>;
  kernel<<<grid, kThreads, 0, stream>>>(a, map, v_warps);
  return cudaGetLastError();
}

}  // namespace nvkv
