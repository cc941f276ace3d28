// combine.cu -- merge the split-K partial results of nvkv_decode_attn.
//
// Each split s of a (sequence, kv-head) pair left, per query row, the
// normalised partial output o_s and lse2_s = base-2 log-sum-exp of its
// scaled scores (-inf when the row saw no key in that split).  The exact
// softmax over the union of the splits is
//     L = max_s lse2_s,  w_s = 2^(lse2_s - L),  out = sum_s w_s o_s / sum_s w_s,
// rounded once to bf16.  One warp per query row; each lane owns D/32
// channels.
#include "score_mod.cuh"
#include "sm100.cuh"

namespace nvkv {

__global__ void __launch_bounds__(256)
combine_kernel(const int32_t *__restrict__ kv_lens, int B, int Hkv, int T, int Hq, int D, int S,
               const float *__restrict__ ws_o, const float *__restrict__ ws_lse,
               __nv_bfloat16 *__restrict__ out) {
  const int G = Hq / Hkv;
  const int R = T * G;
  const long wid = ((long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= (long)B * Hkv * R) return;
  const int bh = (int)(wid / R), r = (int)(wid % R);
  const int b = bh / Hkv, h = bh % Hkv;
  const int t = r / G, g = r % G;
  const int dpl = D / 32;
  __nv_bfloat16 *dst = out + ((size_t)(b * T + t) * Hq + h * G + g) * D + lane * dpl;

  int64_t U = 0, pair_start = 0;
  int units = 0;
  for (int bb = 0; bb < B; ++bb) {
    const int ub = units_of_len(kv_lens[bb]);
    if (bb == b) {
      pair_start = U + (int64_t)h * ub;
      units = ub;
    }
    U += (int64_t)ub * Hkv;
  }
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  float wsum = 0.f;
  if (units > 0) {
    const int64_t c0 = range_of_unit(pair_start, U, S);
    const int64_t c1 = range_of_unit(pair_start + units - 1, U, S);
    // A range that owns no unit (possible only when U < S) wrote nothing.
    const bool all_own_units = U >= S;
    // The lse of up to 32 ranges at a time, one per lane; their max.
    float L = -INFINITY;
    for (int64_t cb = c0; cb <= c1; cb += 32) {
      const int64_t c = cb + lane;
      if (c <= c1 && (all_own_units || range_begin(c, U, S) != range_begin(c + 1, U, S)))
        L = fmaxf(L, ws_lse[(size_t)(c + bh) * R + r]);
    }
    L = warp_max(L);
    if (L > -INFINITY) {
      for (int64_t cb = c0; cb <= c1; cb += 32) {
        const int64_t c = cb + lane;
        float w = 0.f;  // weight of range c; 0 for ranges without keys of this row
        if (c <= c1 && (all_own_units || range_begin(c, U, S) != range_begin(c + 1, U, S))) {
          const float lse = ws_lse[(size_t)(c + bh) * R + r];
          if (lse > -INFINITY) w = exp2f(lse - L);
        }
        const int n = c1 - cb + 1 < 32 ? (int)(c1 - cb + 1) : 32;
        for (int k = 0; k < n; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, k);
          if (wk == 0.f) continue;  // warp-uniform
          wsum += wk;
          const float *o = ws_o + ((size_t)(cb + k + bh) * R + r) * (size_t)D + lane * dpl;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < dpl) acc[i] = fmaf(wk, o[i], acc[i]);
        }
      }
    }
  }
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < dpl) dst[i] = __float2bfloat16_rn(acc[i] * inv);
}

cudaError_t launch_combine(const nvkv_seqs &s, const void *ws_o, const void *ws_lse, int T,
                           int Hq, int Hkv, int D, int S, void *out, cudaStream_t stream) {
  const int R = T * (Hq / Hkv);
  const long warps = (long)s.batch * Hkv * R;
  const int threads = 256;
  const long blocks = (warps * 32 + threads - 1) / threads;
  combine_kernel<<<(unsigned)blocks, threads, 0, stream>>>(
      s.kv_lens, s.batch, Hkv, T, Hq, D, S, static_cast<const float *>(ws_o),
      static_cast<const float *>(ws_lse), static_cast<__nv_bfloat16 *>(out));
  return cudaGetLastError();
}

// The merge of the masked attention (nvkv_decode_attn_mod): the same
// arithmetic, over the units that the queries can see.  kW warps share a row:
// a row of a single long sequence is cut into as many as half the splits of
// the GPU, and one warp walking them, one dependent load after the other,
// took 27 us of a 35 us step (32 ranges of 4,096 tokens, head_dim 128); now
// 5.5 us, most of it the launch's own latency.  Few splits a row (a batch)
// leave each warp a row of its own.  Each warp
// sums the splits w, w + kW, ...; the warps' sums are added in order, so the
// result does not depend on timing.  Started while the attention kernel
// runs (programmatic dependent launch): the split plan is worked out before
// the wait for its partial results.
constexpr int kMergeThreads = 256;

template <int kW>
__global__ void __launch_bounds__(kMergeThreads)
combine_mod_kernel(const int32_t *__restrict__ kv_lens, int B, int Hkv, int T, int Hq, int D, int S,
                   const float *__restrict__ ws_o, const float *__restrict__ ws_lse,
                   __nv_bfloat16 *__restrict__ out, ScoreMod mod) {
  constexpr int kRows = kMergeThreads / 32 / kW;  // rows of a block
  __shared__ float s_acc[kMergeThreads / 32][256];
  __shared__ float s_w[kMergeThreads / 32];
  const int G = Hq / Hkv, R = T * G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % kW;
  const int64_t row = (int64_t)blockIdx.x * kRows + warp / kW;
  const bool live = row < (int64_t)B * Hkv * R;
  const int bh = live ? (int)(row / R) : 0, r = live ? (int)(row % R) : 0;
  const int b = bh / Hkv, h = bh % Hkv;
  // The pair's units and the units before it, 32 sequences at a time.
  int64_t U = 0, before = 0;
  for (int bb = lane; bb < B; bb += 32) {
    const int64_t n = mod.units(kv_lens, bb, T);
    U += n;
    if (bb < b) before += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    U += __shfl_xor_sync(0xffffffffu, U, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  U *= Hkv;
  const int units = live ? mod.units(kv_lens, b, T) : 0;
  const int64_t pair_start = before * Hkv + (int64_t)h * units;
  // (the masked attention deals U units to min(S, U) ranges: none is empty)
  const int64_t Se = split_ranges(U, S);
  int64_t c0 = 0, c1 = -1;
  if (units > 0) {
    c0 = range_of_unit_mod(pair_start, U, Se);
    c1 = range_of_unit_mod(pair_start + units - 1, U, Se);
  }
  sm100::grid_dependency_wait();
  ws_o = sm100::after_wait(ws_o);
  ws_lse = sm100::after_wait(ws_lse);
  sm100::launch_dependents();  // (not before: the attention's SMs are free now)

  const float *lse = ws_lse + (size_t)bh * R + r;
  float mx = -INFINITY;
  bool odd = false;  // a NaN among them: the row's query is not finite
  for (int64_t c = c0 + lane; c <= c1; c += 32) {
    const float v = lse[(size_t)c * R];
    mx = fmaxf(mx, v);
    odd |= isnan(v);
  }
  mx = warp_max(mx);
  odd = __any_sync(0xffffffffu, odd);
  const int dpl = D / 32;  // channels of a lane: 4 or 8
  float acc[8], wsum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  if (mx > -INFINITY || odd) {
    // 32 of this warp's ranges at a time, their weights one a lane
    for (int64_t cb = c0 + sub; cb <= c1; cb += 32 * kW) {
      const int64_t mine = cb + (int64_t)lane * kW;
      const float my = mine <= c1 ? exp2f(lse[(size_t)mine * R] - mx) : 0.f;  // (2^-inf = 0)
      const int n = (int)min((int64_t)32, (c1 - cb) / kW + 1);
#pragma unroll 4
      for (int k = 0; k < n; ++k) {  // warp-uniform
        const float w = __shfl_sync(0xffffffffu, my, k);
        const float *o =
            ws_o + ((size_t)(cb + k * kW + bh) * R + r) * (size_t)D + lane * dpl;
        // (a range that saw no key of the row wrote zeros)
        const float4 a = *reinterpret_cast<const float4 *>(o);
        acc[0] = fmaf(w, a.x, acc[0]), acc[1] = fmaf(w, a.y, acc[1]);
        acc[2] = fmaf(w, a.z, acc[2]), acc[3] = fmaf(w, a.w, acc[3]);
        if (dpl == 8) {
          const float4 e = *reinterpret_cast<const float4 *>(o + 4);
          acc[4] = fmaf(w, e.x, acc[4]), acc[5] = fmaf(w, e.y, acc[5]);
          acc[6] = fmaf(w, e.z, acc[6]), acc[7] = fmaf(w, e.w, acc[7]);
        }
        wsum += w;
      }
    }
  }
  if constexpr (kW > 1) {
    for (int i = 0; i < dpl; ++i) s_acc[warp][lane * dpl + i] = acc[i];
    if (lane == 0) s_w[warp] = wsum;
    __syncthreads();
    if (sub != 0) return;
    for (int w = 1; w < kW; ++w) {
      wsum += s_w[warp + w];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < dpl) acc[i] += s_acc[warp + w][lane * dpl + i];
    }
  }
  if (!live) return;
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
  const int t = r / G, g = r % G;
  __nv_bfloat16 *dst = out + ((size_t)(b * T + t) * Hq + h * G + g) * D + lane * dpl;
  uint32_t ow[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    ow[i] = *reinterpret_cast<const uint32_t *>(&v);
  }
  if (dpl == 8)
    *reinterpret_cast<uint4 *>(dst) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
  else
    *reinterpret_cast<uint2 *>(dst) = make_uint2(ow[0], ow[1]);
}

cudaError_t launch_combine_mod(const nvkv_seqs &s, const float *ws_o, const float *ws_lse, int T,
                               int Hq, int Hkv, int D, int S, void *out, cudaStream_t stream,
                               const ScoreMod &mod) {
  const int64_t rows = (int64_t)s.batch * Hkv * T * (Hq / Hkv);
  // ranges a pair can span: its share of the splits and one at either end
  const bool shared = S / ((int64_t)s.batch * Hkv) + 2 > 4;
  const int per_block = shared ? 1 : kMergeThreads / 32;
  const DependentLaunch launch(dim3((unsigned)((rows + per_block - 1) / per_block)), kMergeThreads,
                               0, stream, true);
  return cudaLaunchKernelEx(&launch.cfg, shared ? combine_mod_kernel<8> : combine_mod_kernel<1>,
                            s.kv_lens, s.batch, Hkv, T, Hq, D, S, ws_o, ws_lse,
                            static_cast<__nv_bfloat16 *>(out), mod);
}

}  // namespace nvkv
