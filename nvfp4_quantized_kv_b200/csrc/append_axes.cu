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
//  * V warps take one page of one kv-head (two at head_dim 128), 8 head_dim
//    elements a lane, and gather the nibbles of all new slots in registers:
//    V is stored transposed, so a page that is new as a whole leaves as 64
//    contiguous bytes a lane; otherwise only the bytes of slot pairs with a
//    new slot are written (the other nibble of such a byte is kept).
#include "nvkv_common.cuh"

namespace nvkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeadsPerWarp = 8;
constexpr int kMaxAxes = 4;

struct AxisMap {
  uint8_t axis[128];  // of each pair
};

__device__ __forceinline__ void load8(const __nv_bfloat16 *src, float (&x)[8]) {
  const uint4 r = __ldg(reinterpret_cast<const uint4 *>(src));
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16 *dst, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&r);
  }
  *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float amax8(const float (&x)[8]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
  return a;
}

// The codes of 8 elements under a scale byte (element 0 in bits 0..3).
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], uint8_t scale) {
  uint32_t c = 0;
  if (scale) {
    const float s = e4m3_to_float(scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) c |= e2m1_code(x[i], s) << (4 * i);
  }
  return c;
}

// Whether row `row` has a table row on every axis.
__device__ __forceinline__ bool positions_ok(const int32_t *pos, int axes, int total, int row,
                                             int max_pos) {
  bool ok = true;
  for (int a = 0; a < axes; ++a) {
    const int p = pos[(size_t)a * total + row];
    ok &= p >= 0 && p < max_pos;
  }
  return ok;
}

struct Args {
  uint8_t *pool;
  int num_pages, Hkv, D;
  const int32_t *page_table;
  int max_pages;
  const int32_t *kv_lens;
  int max_kv_len;
  const __nv_bfloat16 *k, *v, *q;  // q null: no queries
  __nv_bfloat16 *q_out;
  int Hq;
  const int32_t *cu_new;
  int total_new, max_new;
  const float *cs;
  int max_pos, rotary_dim;
  const int32_t *positions;
  int axes;
  int32_t *err;
};

__global__ void __launch_bounds__(kThreads)
append_axes_kernel(const Args a, const __grid_constant__ AxisMap map, int row_warps) {
  const int b = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int wid = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int D = a.D;

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

  if (wid < row_warps) {
    // ---------------------------------------------- K heads or query heads
    const int kchunks = (a.Hkv + kHeadsPerWarp - 1) / kHeadsPerWarp;
    const int qchunks = a.q ? (a.Hq + kHeadsPerWarp - 1) / kHeadsPerWarp : 0;
    const int i = wid / (kchunks + qchunks), chunk = wid % (kchunks + qchunks);
    if (i >= n) return;
    const int row = row0 + i, pos = first + i;
    const bool is_q = chunk >= kchunks;
    const int page = page_at(pos);
    if (page < 0) {
      if (chunk == 0 && lane == 0) report(a.err, NVKV_DEVERR_PAGE_ID);
      if (!is_q) return;
    }
    if (!positions_ok(a.positions, a.axes, a.total_new, row, a.max_pos)) {
      if (chunk == 0 && lane == 0) report(a.err, NVKV_DEVERR_LENGTH);
      return;
    }
    const int lanes = D / 16;                    // of a head
    const int l = lane % lanes, sub = lane / lanes;
    const int half = a.rotary_dim / 2;
    const bool turn = 8 * l < half;
    // elements of this lane: [e0, e0 + 8) and [e1, e1 + 8)
    const int e0 = turn ? 8 * l : a.rotary_dim + 16 * (l - half / 8);
    const int e1 = turn ? half + 8 * l : e0 + 8;
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = 1.f, s[e] = 0.f;
      if (turn) {
        const int p = a.positions[(size_t)map.axis[8 * l + e] * a.total_new + row];
        const float2 v = *reinterpret_cast<const float2 *>(
            a.cs + (size_t)p * a.rotary_dim + 2 * (8 * l + e));
        c[e] = v.x, s[e] = v.y;
      }
    }
    const int heads = is_q ? a.Hq : a.Hkv;
    const int h0 = (is_q ? chunk - kchunks : chunk) * kHeadsPerWarp;
    const int h1 = min(h0 + kHeadsPerWarp, heads);
    const __nv_bfloat16 *src = (is_q ? a.q : a.k) + (size_t)row * heads * D;
#pragma unroll 2
    for (int hb = h0; hb < h1; hb += 32 / lanes) {  // warp-uniform
      const int h = hb + sub;
      const bool live = h < h1;
      float x[8], y[8];
      if (live) {
        load8(src + (size_t)h * D + e0, x);
        load8(src + (size_t)h * D + e1, y);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = y[e] = 0.f;
      }
      if (turn) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float ys = __fmul_rn(y[e], s[e]), xs = __fmul_rn(x[e], s[e]);
          x[e] = fmaf(x[e], c[e], -ys);
          y[e] = fmaf(y[e], c[e], xs);
        }
      }
      if (is_q) {
        if (live) {
          store8(a.q_out + ((size_t)row * heads + h) * D + e0, x);
          store8(a.q_out + ((size_t)row * heads + h) * D + e1, y);
        }
        continue;
      }
      // group maxima: a rotated group is this lane and its neighbour
      float ax = amax8(x), ay = amax8(y);
      const float nx = __shfl_xor_sync(0xffffffffu, ax, 1), ny = __shfl_xor_sync(0xffffffffu, ay, 1);
      ax = turn ? fmaxf(ax, nx) : fmaxf(ax, ay);
      ay = turn ? fmaxf(ay, ny) : ax;
      const uint8_t sx = scale_byte_of_amax(ax), sy = scale_byte_of_amax(ay);
      const uint32_t cx = codes8(x, sx), cy = codes8(y, sy);
      if (!live) continue;
      const int slot = pos % kPageTokens;
      uint8_t *blk = a.pool + ((size_t)page * a.Hkv + h) * head_bytes(D);
      *reinterpret_cast<uint32_t *>(blk + kc_off(D) + slot * (D / 2) + e0 / 2) = cx;
      *reinterpret_cast<uint32_t *>(blk + kc_off(D) + slot * (D / 2) + e1 / 2) = cy;
      uint8_t *ks = blk + ks_off(D) + slot * (D / 16);
      if (turn) {
        // even lane: the x group's scale, odd lane: the y group's
        if (l & 1)
          ks[e1 / 16] = sy;
        else
          ks[e0 / 16] = sx;
      } else {
        ks[e0 / 16] = sx;
      }
    }
    return;
  }

  // ------------------------------------------------------------------- V
  const int lanes = D / 8;
  const int l = lane % lanes;
  const int64_t ph = (int64_t)(wid - row_warps) * (32 / lanes) + lane / lanes;
  const int h = (int)(ph % a.Hkv);
  const int64_t pi = first / kPageTokens + ph / a.Hkv;
  bool live = pi * kPageTokens < len;
  const int p0 = live ? (int)pi * kPageTokens : 0;
  const int page = live ? page_at(p0) : -1;
  live = page >= 0;  // (reported by the row warps)
  // New slots of the page: inside [first, len), with a table row.
  uint32_t fresh = 0;
  {
    const int hl = lane & 15;
    const int pos = p0 + hl;
    bool ok = live && pos >= first && pos < len;
    if (ok) ok = positions_ok(a.positions, a.axes, a.total_new, row0 + pos - first, a.max_pos);
    // the unit's 16 slots: at head_dim 256 both half-warps vote on the same
    // page, at 128 each on its own
    fresh = (__ballot_sync(0xffffffffu, ok) >> (lane & 16)) & 0xffffu;
  }
  uint8_t *blk = a.pool + ((size_t)(live ? page : 0) * a.Hkv + h) * head_bytes(D);
  const __nv_bfloat16 *src =
      a.v + ((int64_t)row0 + p0 - first) * (int64_t)a.Hkv * D + (size_t)h * D + 8 * l;
  uint32_t w[16];  // [element i][slots 0..7, slots 8..15] at 2 * i
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = 0u;
  uint32_t sc[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int sl = 0; sl < kPageTokens; ++sl) {
    const bool is_new = (fresh >> sl) & 1u;
    if (!__any_sync(0xffffffffu, is_new)) continue;
    float x[8];
    if (is_new) {
      load8(src + (int64_t)sl * a.Hkv * D, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
    }
    float ax = amax8(x);
    ax = fmaxf(ax, __shfl_xor_sync(0xffffffffu, ax, 1));
    const uint8_t sb = scale_byte_of_amax(ax);
    const uint32_t c = codes8(x, sb);
    sc[sl >> 2] |= (uint32_t)sb << (8 * (sl & 3));
#pragma unroll
    for (int e = 0; e < 8; ++e)
      w[2 * e + (sl >> 3)] |= ((c >> (4 * e)) & 15u) << (4 * (sl & 7));
  }
  if (fresh == 0) return;
  uint8_t *vc = blk + vc_off(D) + 64 * l;
  uint8_t *vs = blk + vs_off(D) + (l >> 1) * kPageTokens;
  if (fresh == 0xffffu) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<uint4 *>(vc)[i] =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    if ((l & 1) == 0) *reinterpret_cast<uint4 *>(vs) = make_uint4(sc[0], sc[1], sc[2], sc[3]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {  // slot pair (2j, 2j + 1): byte j of each element
    const uint32_t two = (fresh >> (2 * j)) & 3u;
    if (two == 0) continue;
    const uint32_t keep = two == 3u ? 0u : two == 1u ? 0xf0u : 0x0fu;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t byte = (w[2 * e + (j >> 2)] >> (8 * (j & 3))) & 0xffu;
      if (keep) byte |= vc[8 * e + j] & keep;
      vc[8 * e + j] = (uint8_t)byte;
    }
    if ((l & 1) == 0) {
      if (two & 1u) vs[2 * j] = (uint8_t)(sc[j >> 1] >> (16 * (j & 1)));
      if (two & 2u) vs[2 * j + 1] = (uint8_t)(sc[j >> 1] >> (16 * (j & 1) + 8));
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
  return (pages * c.num_kv_heads + per_warp - 1) / per_warp;
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
  a.pool = c.pool, a.num_pages = c.num_pages, a.Hkv = c.num_kv_heads, a.D = c.head_dim;
  a.page_table = s.page_table, a.max_pages = s.max_pages_per_seq;
  a.kv_lens = s.kv_lens, a.max_kv_len = s.max_kv_len;
  a.k = static_cast<const __nv_bfloat16 *>(k_new);
  a.v = static_cast<const __nv_bfloat16 *>(v_new);
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.q_out = static_cast<__nv_bfloat16 *>(q_out);
  a.Hq = Hq, a.cu_new = cu_new, a.total_new = total_new, a.max_new = max_new;
  a.cs = cs, a.max_pos = max_pos, a.rotary_dim = rotary_dim;
  a.positions = positions, a.axes = axes, a.err = s.err_word;
  AxisMap map{};
  for (int i = 0; i < rotary_dim / 2; ++i) map.axis[i] = axis_of_pair[i];
  const int row_warps = (int)row_warps_of(c, max_new, Hq, q != nullptr);
  const int64_t warps = row_warps + v_warps_of(c, max_new);
  const dim3 grid((unsigned)((warps + kWarps - 1) / kWarps), (unsigned)s.batch);
  append_axes_kernel<<<grid, kThreads, 0, stream>>>(a, map, row_warps);
  return cudaGetLastError();
}

}  // namespace nvkv
