// rows.cu -- nvkv_read_rows: cached K/V rows back as bf16 [rows][Hkv][D].
//
// An NVFP4 value E2M1 * E4M3 has at most 6 significant bits and lies in
// [2^-10, 2688], so it is a bf16 number and the read is exact; a K8V4 K value
// E4M3 * scale (fp32) is rounded once.
//
// Bound by HBM: 1.125*D bytes of cache in and 4*D out per token and kv-head
// (K8V4: 1.5625*D + 4 in).  D/8 lanes ("a unit": half a warp at head_dim 128)
// take the 16 slots of one page and kv-head, K or V, 8 head_dim elements a
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
#include <type_traits>

#include "nvkv_common.cuh"

namespace nvkv {
namespace {

constexpr int kThreads = 256;

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

template <class L>
__global__ void __launch_bounds__(kThreads)
read_rows_kernel(const uint8_t *__restrict__ pool, int num_pages, int Hkv, int D,
                 const int32_t *__restrict__ page_table, int max_pages,
                 const int32_t *__restrict__ kv_lens, int max_kv_len,
                 const int32_t *__restrict__ starts, const int32_t *__restrict__ cu_rows,
                 int total_rows, int max_rows, __nv_bfloat16 *__restrict__ k_out,
                 __nv_bfloat16 *__restrict__ v_out, int32_t *err) {
  const int b = blockIdx.y;
  const int lanes = D / 8;  // lanes of a unit: 16 or 32
  const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / lanes;
  const int l = threadIdx.x % lanes;
  const int row0 = cu_rows[b], n = cu_rows[b + 1] - row0;
  if (n <= 0) return;
  const int first = starts[b], len = kv_lens[b];
  if (row0 < 0 || row0 > total_rows - n || n > max_rows || first < 0 || first > len - n ||
      len > max_kv_len || len > max_pages * kPageTokens) {
    if (unit == 0 && l == 0) report(err, NVKV_DEVERR_LENGTH);
    return;
  }
  // A warp's units (one, or two at head_dim 128) are consecutive (page of the
  // row range, kv-head) blocks, all K or all V.
  const int per_warp = 32 / lanes;
  const int64_t w2 = unit / per_warp;
  const bool is_v = w2 & 1;
  const int64_t ph = (w2 >> 1) * per_warp + unit % per_warp;
  const int h = (int)(ph % Hkv);
  const int64_t pi = first / kPageTokens + ph / Hkv;
  if (pi * kPageTokens >= first + n) return;
  const int page = page_table[(size_t)b * max_pages + pi];
  if (page < 0 || page >= num_pages) {
    if (l == 0) report(err, NVKV_DEVERR_PAGE_ID);
    return;
  }
  const uint8_t *blk = pool + ((size_t)page * Hkv + h) * L::head(D);
  // slots [s0, s1) of the page are asked for; row of slot s: row0 + p0 + s
  const int p0 = (int)pi * kPageTokens - first;
  const int s0 = max(0, -p0), s1 = min(kPageTokens, n - p0);
  const size_t stride = (size_t)Hkv * D;
  __nv_bfloat16 *dst =
      (is_v ? v_out : k_out) + ((int64_t)row0 + p0) * (int64_t)stride + (size_t)h * D + 8 * l;
  if (is_v) {
    const uint4 *src = reinterpret_cast<const uint4 *>(blk + L::vc(D) + 64 * l);
    uint32_t w[16];  // [element i][slots 0..7, slots 8..15] at 2 * i
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = __ldg(src + i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
    const uint4 sc4 =
        __ldg(reinterpret_cast<const uint4 *>(blk + L::vs(D) + (l >> 1) * kPageTokens));
    const uint32_t scw[4] = {sc4.x, sc4.y, sc4.z, sc4.w};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t a = scw[2 * half], c = scw[2 * half + 1];
      // the scales of slots (t, t + 4) of this half
      const uint32_t sp[4] = {scale_pair(__byte_perm(a, c, 0x40)), scale_pair(__byte_perm(a, c, 0x51)),
                              scale_pair(__byte_perm(a, c, 0x62)), scale_pair(__byte_perm(a, c, 0x73))};
      auto slots = [&](auto tc) {
        constexpr int t = decltype(tc)::value;
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = mul_bf16x2(
              mul_bf16x2(bf16_code_pair<t>(w[4 * i + half]), kTwo120), sp[t]);
          const uint32_t y = mul_bf16x2(
              mul_bf16x2(bf16_code_pair<t>(w[4 * i + 2 + half]), kTwo120), sp[t]);
          lo[i] = __byte_perm(x, y, 0x5410);
          hi[i] = __byte_perm(x, y, 0x7632);
        }
        const int s = 8 * half + t;
        if (s >= s0 && s < s1) store_row(dst + (int64_t)s * stride, lo);
        if (s + 4 >= s0 && s + 4 < s1) store_row(dst + (int64_t)(s + 4) * stride, hi);
      };
      slots(std::integral_constant<int, 0>{});
      slots(std::integral_constant<int, 1>{});
      slots(std::integral_constant<int, 2>{});
      slots(std::integral_constant<int, 3>{});
    }
  } else if constexpr (L::kK8) {
#pragma unroll 4
    for (int s = s0; s < s1; ++s) {
      const uint2 w = __ldg(reinterpret_cast<const uint2 *>(blk + (size_t)s * D + 8 * l));
      const float sc = __ldg(reinterpret_cast<const float *>(blk + k8_ks_off(D) + 4 * s));
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t h2[2];
        e4m3x4_to_f16x2x2(k ? w.y : w.x, h2);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f = f16x2_to_float2(h2[j]);
          const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * sc, f.y * sc);
          o[2 * k + j] = *reinterpret_cast<const uint32_t *>(&r);
        }
      }
      store_row(dst + (int64_t)s * stride, o);
    }
  } else {
#pragma unroll 8
    for (int s = s0; s < s1; ++s) {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(blk + s * (D / 2) + 4 * l));
      const uint32_t sb = __ldg(blk + ks_off(D) + s * (D / 16) + (l >> 1));
      const uint32_t sp = scale_pair(sb | (sb << 8));
      const uint32_t x[4] = {
          mul_bf16x2(mul_bf16x2(bf16_code_pair<0>(w), kTwo120), sp),
          mul_bf16x2(mul_bf16x2(bf16_code_pair<1>(w), kTwo120), sp),
          mul_bf16x2(mul_bf16x2(bf16_code_pair<2>(w), kTwo120), sp),
          mul_bf16x2(mul_bf16x2(bf16_code_pair<3>(w), kTwo120), sp)};
      const uint32_t o[4] = {__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410),
                             __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632)};
      store_row(dst + (int64_t)s * stride, o);
    }
  }
}

}  // namespace

// Blocks that max_rows rows of one sequence can need (a range may start and
// end inside a page).
int64_t read_rows_blocks(const nvkv_cache &c, int max_rows) {
  const int64_t pages = ((int64_t)max_rows + 2 * kPageTokens - 2) / kPageTokens;
  const int per_warp = 256 / c.head_dim;  // (page, kv-head) blocks of a warp
  const int64_t warps = (pages * c.num_kv_heads + per_warp - 1) / per_warp * 2;
  return (warps * 32 + kThreads - 1) / kThreads;
}

// k8: the pool is in the K8V4 layout (else NVFP4).
cudaError_t launch_read_rows(const nvkv_cache &c, const nvkv_seqs &s, const int32_t *starts,
                             const int32_t *cu_rows, int total_rows, int max_rows, void *k_out,
                             void *v_out, cudaStream_t stream, bool k8) {
  const dim3 grid((unsigned)read_rows_blocks(c, max_rows), (unsigned)s.batch);
  auto kernel = k8 ? read_rows_kernel<K8v4Layout> : read_rows_kernel<Nvfp4Layout>;
  kernel<<<grid, kThreads, 0, stream>>>(
      c.pool, c.num_pages, c.num_kv_heads, c.head_dim, s.page_table, s.max_pages_per_seq,
      s.kv_lens, s.max_kv_len, starts, cu_rows, total_rows, max_rows,
      static_cast<__nv_bfloat16 *>(k_out), static_cast<__nv_bfloat16 *>(v_out), s.err_word);
  return cudaGetLastError();
}

}  // namespace nvkv
