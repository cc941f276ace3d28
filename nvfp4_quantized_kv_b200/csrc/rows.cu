// rows.cu -- nvkv_read_rows: cached K/V rows back as bf16 [rows][Hkv][D].
//
// An NVFP4 value E2M1 * E4M3 has at most 6 significant bits and lies in
// [2^-10, 2688], so it is a bf16 number and the read is exact; a K8V4 K value
// E4M3 * scale (fp32) is rounded once.
//
// Bound by HBM: 1.125*D bytes of cache in and 4*D out per token and kv-head
// (K8V4: 1.5625*D + 4 in).  D/8 lanes ("a unit": half a warp at head_dim 128)
// take the 16 slots of a page and kv-head, K or V, 8 head_dim elements a
// lane:
//  * a K row is D/2 consecutive bytes, 4 a lane, and leaves as 16 bytes a lane;
//  * V is stored transposed, 8 bytes for the 16 slots of one head_dim
//    element: a lane loads the 64 consecutive bytes of its 8 elements, builds
//    the rows in registers and stores 16 bytes of each, so every store of the
//    unit is one contiguous row and nothing goes through shared memory.
// Codes become bf16 with integer operations (a conversion instruction runs
// at a fraction of the rate): the bits (mag << 6) | (sign << 15) are
// E2M1 * 2^-126 as bf16, and two exact multiplies bring in 2^120 and the
// scale times 2^6.
//
// Measured (NVFP4): 130,001 rows of 4 kv-heads at head_dim 256, 4 sequences:
// 119 us = 5,730 GB/s, 0.87 of the measured copy rate; 994 rows of 2 kv-heads
// at head_dim 128: 3.5 us, the launch and three dependent loads.
#include <climits>

#include "nvkv_common.cuh"

namespace nvkv {
namespace {

constexpr int kThreads = 256;

// Blocks that max_rows rows of one sequence can need (a range may start and
// end inside a page).
int64_t read_rows_blocks(const nvkv_cache &c, int max_rows, int pages_per_unit) {
  const int64_t pages = ((int64_t)max_rows + 2 * kPageTokens - 2) / kPageTokens;
  const int per_warp = 256 / c.head_dim;  // units of a warp
  const int64_t units = (pages + pages_per_unit - 1) / pages_per_unit * c.num_kv_heads;
  return ((units + per_warp - 1) / per_warp * 2 * 32 + kThreads - 1) / kThreads;
}

// Elements t (low half) and t + 4 (high half) of a word of 8 codes, as bf16
// times 2^-126.
template <int t>
__device__ __forceinline__ uint32_t bf16_code_pair(uint32_t w) {
  const uint32_t a = t < 2 ? (w << (6 - 4 * t)) : (w >> (4 * t - 6));
  return (a & 0x02000200u) * 64u + (a & 0x01C001C0u);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

constexpr uint32_t kTwo120 = 0x7B807B80u;  // bf16 pair (2^120, 2^120)

// Two E4M3 bytes (low first) -> bf16 pair of their values times 2^6, exact.
__device__ __forceinline__ uint32_t scale_pair(uint32_t two) {
  const float2 f = f16x2_to_float2(e4m3x2_to_f16x2(two));
  return __byte_perm(__float_as_uint(f.x * 64.f), __float_as_uint(f.y * 64.f), 0x7632);
}

__device__ __forceinline__ void store_row(__nv_bfloat16 *dst, const uint32_t (&w)[4]) {
  *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

// What a lane reads of one page block: the codes and scales of its 8
// elements in all 16 slots.
struct PageV {
  uint32_t w[16];  // [element i][slots 0..7, slots 8..15] at 2 * i
  uint32_t sc[4];  // the 16 slots' scale bytes

  template <class L>
  __device__ __forceinline__ void load(const uint8_t *blk, int D, int l) {
    const uint4 *src = reinterpret_cast<const uint4 *>(blk + L::vc(D) + 64 * l);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = __ldg(src + i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(blk + L::vs(D) + (l >> 1) * kPageTokens));
    sc[0] = v.x, sc[1] = v.y, sc[2] = v.z, sc[3] = v.w;
  }

  // Slots [s0, s1) to the rows at dst (slot 0) with the given stride.
  __device__ __forceinline__ void store(__nv_bfloat16 *dst, int64_t stride, int s0, int s1) const {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t a = sc[2 * half], c = sc[2 * half + 1];
      slots<0>(dst, stride, s0, s1, half, scale_pair(__byte_perm(a, c, 0x40)));
      slots<1>(dst, stride, s0, s1, half, scale_pair(__byte_perm(a, c, 0x51)));
      slots<2>(dst, stride, s0, s1, half, scale_pair(__byte_perm(a, c, 0x62)));
      slots<3>(dst, stride, s0, s1, half, scale_pair(__byte_perm(a, c, 0x73)));
    }
  }

  // Slots 8 * half + t and 8 * half + t + 4, whose scales are the pair sp.
  template <int t>
  __device__ __forceinline__ void slots(__nv_bfloat16 *dst, int64_t stride, int s0, int s1,
                                        int half, uint32_t sp) const {
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x =
          mul_bf16x2(mul_bf16x2(bf16_code_pair<t>(w[4 * i + half]), kTwo120), sp);
      const uint32_t y =
          mul_bf16x2(mul_bf16x2(bf16_code_pair<t>(w[4 * i + 2 + half]), kTwo120), sp);
      lo[i] = __byte_perm(x, y, 0x5410);
      hi[i] = __byte_perm(x, y, 0x7632);
    }
    const int sl = 8 * half + t;
    if (sl >= s0 && sl < s1) store_row(dst + sl * stride, lo);
    if (sl + 4 >= s0 && sl + 4 < s1) store_row(dst + (sl + 4) * stride, hi);
  }
};

struct PageK {
  uint32_t w[16];   // [slot]: 8 codes
  uint32_t sb[16];  // [slot]: the group's scale byte

  template <class L>
  __device__ __forceinline__ void load(const uint8_t *blk, int D, int l) {
#pragma unroll
    for (int sl = 0; sl < kPageTokens; ++sl) {
      w[sl] = __ldg(reinterpret_cast<const uint32_t *>(blk + sl * (D / 2) + 4 * l));
      sb[sl] = __ldg(blk + ks_off(D) + sl * (D / 16) + (l >> 1));
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *dst, int64_t stride, int s0, int s1) const {
#pragma unroll
    for (int sl = 0; sl < kPageTokens; ++sl) {
      const uint32_t sp = scale_pair(sb[sl] | (sb[sl] << 8));
      const uint32_t x[4] = {mul_bf16x2(mul_bf16x2(bf16_code_pair<0>(w[sl]), kTwo120), sp),
                             mul_bf16x2(mul_bf16x2(bf16_code_pair<1>(w[sl]), kTwo120), sp),
                             mul_bf16x2(mul_bf16x2(bf16_code_pair<2>(w[sl]), kTwo120), sp),
                             mul_bf16x2(mul_bf16x2(bf16_code_pair<3>(w[sl]), kTwo120), sp)};
      const uint32_t o[4] = {__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410),
                             __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632)};
      if (sl >= s0 && sl < s1) store_row(dst + sl * stride, o);
    }
  }
};

// K8V4: one E4M3 byte an element, one fp32 scale a row.
struct PageK8 {
  uint2 w[16];
  float sc[16];

  template <class L>
  __device__ __forceinline__ void load(const uint8_t *blk, int D, int l) {
#pragma unroll
    for (int sl = 0; sl < kPageTokens; ++sl) {
      w[sl] = __ldg(reinterpret_cast<const uint2 *>(blk + sl * D + 8 * l));
      sc[sl] = __ldg(reinterpret_cast<const float *>(blk + k8_ks_off(D) + 4 * sl));
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *dst, int64_t stride, int s0, int s1) const {
#pragma unroll
    for (int sl = 0; sl < kPageTokens; ++sl) {
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t h2[2];
        e4m3x4_to_f16x2x2(k ? w[sl].y : w[sl].x, h2);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f = f16x2_to_float2(h2[j]);
          const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * sc[sl], f.y * sc[sl]);
          o[2 * k + j] = *reinterpret_cast<const uint32_t *>(&r);
        }
      }
      if (sl >= s0 && sl < s1) store_row(dst + sl * stride, o);
    }
  }
};

struct Rows {  // the unit's share of a call
  const uint8_t *pool;      // kv-head block of page 0
  int64_t page_bytes;
  int D, l;
  __nv_bfloat16 *dst;       // element 8 * l of slot 0 of the unit's first page
  int64_t stride;           // elements from row to row
  int p0, n;                // row of that slot, rows asked for
};

template <class Page, class L, int kPages>
__device__ __forceinline__ void read_pages(const Rows &r, const int (&pages)[kPages]) {
  Page cur, next;
  if (pages[0] >= 0) cur.template load<L>(r.pool + pages[0] * r.page_bytes, r.D, r.l);
#pragma unroll
  for (int k = 0; k < kPages; ++k) {
    if (k + 1 < kPages && pages[k + 1 < kPages ? k + 1 : 0] >= 0)
      next.template load<L>(r.pool + pages[k + 1 < kPages ? k + 1 : 0] * r.page_bytes, r.D, r.l);
    const int p = r.p0 + k * kPageTokens;
    if (pages[k] >= 0)
      cur.store(r.dst + (int64_t)k * kPageTokens * r.stride, r.stride, max(0, -p),
                min(kPageTokens, r.n - p));
    cur = next;
  }
}

// kPages consecutive pages of one kv-head for each unit; the next page's
// loads are under way while a page is written.
template <class L, int kPages>
__global__ void __launch_bounds__(kThreads)
read_rows_kernel(const uint8_t *__restrict__ pool, int num_pages, int Hkv, int D,
                 const int32_t *__restrict__ page_table, int max_pages,
                 const int32_t *__restrict__ kv_lens, int max_kv_len,
                 const int32_t *__restrict__ starts, const int32_t *__restrict__ cu_rows,
                 int total_rows, int max_rows, __nv_bfloat16 *__restrict__ k_out,
                 __nv_bfloat16 *__restrict__ v_out, int32_t *err) {
  const int b = blockIdx.y;
  const int lanes = D / 8;  // lanes of a unit: 16 or 32
  const unsigned warp = (blockIdx.x * (unsigned)kThreads + threadIdx.x) / 32;
  const int lane = threadIdx.x & 31, l = lane & (lanes - 1);
  const int row0 = cu_rows[b], n = cu_rows[b + 1] - row0;
  const int first = starts[b], len = kv_lens[b];
  if (n <= 0) return;
  if (row0 < 0 || row0 > total_rows - n || n > max_rows || first < 0 || first > len - n ||
      len > max_kv_len || len > max_pages * kPageTokens) {
    if (warp == 0 && lane == 0) report(err, NVKV_DEVERR_LENGTH);
    return;
  }
  // A warp's units (one, or two at head_dim 128) are all K or all V.
  const bool is_v = warp & 1;
  const unsigned unit = D == 256 ? warp >> 1 : (warp >> 1) * 2 + (lane >> 4);
  const unsigned group = unit / (unsigned)Hkv;
  const int h = (int)(unit - group * (unsigned)Hkv);
  const int64_t pi = first / kPageTokens + (int64_t)group * kPages;
  const int64_t end = ((int64_t)first + n + kPageTokens - 1) / kPageTokens;
  if (pi >= end) return;
  int pages[kPages];
  const int32_t *pt = page_table + (size_t)b * max_pages + pi;
#pragma unroll
  for (int k = 0; k < kPages; ++k) pages[k] = pi + k < end ? pt[k] : -1;
#pragma unroll
  for (int k = 0; k < kPages; ++k) {
    if (pi + k < end && (pages[k] < 0 || pages[k] >= num_pages)) {
      if (l == 0) report(err, NVKV_DEVERR_PAGE_ID);
      pages[k] = -1;
    }
  }
  Rows r;
  r.pool = pool + (size_t)h * L::head(D);
  r.page_bytes = (int64_t)Hkv * L::head(D);
  r.D = D, r.l = l, r.n = n;
  r.p0 = (int)pi * kPageTokens - first;
  r.stride = (int64_t)Hkv * D;
  r.dst = (is_v ? v_out : k_out) + ((int64_t)row0 + r.p0) * r.stride + (size_t)h * D + 8 * l;
  if (is_v)
    read_pages<PageV, L, kPages>(r, pages);
  else if constexpr (L::kK8)
    read_pages<PageK8, L, kPages>(r, pages);
  else
    read_pages<PageK, L, kPages>(r, pages);
}

// Pages of a unit: 4, or 1 for calls of less than about two waves of warps,
// whose time is the latency of one unit.
int pages_per_unit(const nvkv_cache &c, const nvkv_seqs &s, int max_rows) {
  const int64_t units = ((int64_t)max_rows + kPageTokens - 1) / kPageTokens * c.num_kv_heads * 2 *
                        s.batch / (256 / c.head_dim);
  return units < 148 * 64 ? 1 : 4;
}

template <class L>
cudaError_t launch_fmt(const nvkv_cache &c, const nvkv_seqs &s, const int32_t *starts,
                       const int32_t *cu_rows, int total_rows, int max_rows, void *k_out,
                       void *v_out, cudaStream_t stream) {
  const int per = pages_per_unit(c, s, max_rows);
  auto kernel = per == 1 ? read_rows_kernel<L, 1> : read_rows_kernel<L, 4>;
  const dim3 grid((unsigned)read_rows_blocks(c, max_rows, per), (unsigned)s.batch);
  kernel<<<grid, kThreads, 0, stream>>>(
      c.pool, c.num_pages, c.num_kv_heads, c.head_dim, s.page_table, s.max_pages_per_seq,
      s.kv_lens, s.max_kv_len, starts, cu_rows, total_rows, max_rows,
      static_cast<__nv_bfloat16 *>(k_out), static_cast<__nv_bfloat16 *>(v_out), s.err_word);
  return cudaGetLastError();
}

}  // namespace

// Whether the kernel's 32-bit warp index holds the call.
bool read_rows_fits(const nvkv_cache &c, int max_rows) {
  return read_rows_blocks(c, max_rows, 1) * (kThreads / 32) <= INT32_MAX;
}

// k8: the pool is in the K8V4 layout (else NVFP4).
cudaError_t launch_read_rows(const nvkv_cache &c, const nvkv_seqs &s, const int32_t *starts,
                             const int32_t *cu_rows, int total_rows, int max_rows, void *k_out,
                             void *v_out, cudaStream_t stream, bool k8) {
  return k8 ? launch_fmt<K8v4Layout>(c, s, starts, cu_rows, total_rows, max_rows, k_out, v_out,
                                     stream)
            : launch_fmt<Nvfp4Layout>(c, s, starts, cu_rows, total_rows, max_rows, k_out, v_out,
                                      stream);
}

}  // namespace nvkv
