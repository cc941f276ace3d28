// prefill_mod.cu -- chunked prefill with modified scores and masks
// (nvkv_prefill_attn_mod) over the NVFP4 paged pool on the 5th-generation
// tensor cores (tcgen05), head_dim 128 and 256.
//
// Per query row i (position p, head hq): x_j = sm_scale q_i.k_j, capped by
// cap * tanh(x / cap), minus slope * |p - j|, over the keys lo_i <= j < hi_i
// of its interval (score_mod.cuh); softmax; times V.
//
// One CTA owns 128 query rows (chunk tokens x GQA heads) of one kv-head and
// streams the 64-token key tiles that any of its rows sees; with a distance
// bias from the newest to the oldest, so that the largest scores come first
// and the running maximum is found in the first tile instead of being raised
// in every one. Q (128 x D, f16) sits in Tensor Memory as the A operand of
// S = Q K^T (N = 64), S is double-buffered there, P (f16) overwrites its own S
// slot as the A operand of O += P V (N = D), O stays in Tensor Memory.
//
// A row of Q is its bf16 values times the power of two that puts the largest
// into [2^14, 2^15): 8 significant bits, so nothing is rounded but elements
// below 2^-31 of that largest one (f16 subnormals; by at most 2^-39 of it), and
// no size of q overflows. sm_scale * log2(e) and the power of two come back as
// one fp32 factor of the row's scores. (sm_scale in Q itself took 11 bits of
// the product, fewer than the plain verify step's two f16 terms, and ended at
// |q * sm_scale| = 45,000.) The rows' maxima and the factor cost 0.4 to 2.6 %:
// long chunk 3.85 -> 3.86 ms, windows 80.2 -> 81.1 us, verify step 46.1 -> 47.3.
//
// Roles, and what set the pace before each of them (clock64 traces, cycles a
// tile at head_dim 256 with a cap):
//  * With one thread for a row's 64 scores, and one such warp on each SM
//    sub-partition, the softmax took 3,900. Two warpgroups share every tile,
//    32 keys each; the two threads of a row agree on its running maximum only
//    when a score may pass it by 2^8, which one barrier of their two warps
//    detects (it also keeps P from overwriting scores not yet read).
//  * K and V have warps of their own (4 and 8: V's 8 take 1,100, 4 took
//    2,700).
//  * One thread for all MMAs, polling for whichever could go, held a tile's
//    value MMAs back behind the next tile's scores (issuing a batch blocks
//    until it has nearly executed), and with them the S slot that the scores
//    after those wait for: 3,200. Two issuing threads: 2,700. Issued by
//    converged warps instead (mma_f16_ts_warp), the scores of a tile issue in
//    900 cycles, not 1,850: 2,550, of which the softmax is busy 2,300. The
//    MMAs themselves need 800 (scores: 48 cycles an instruction is the least
//    at N = 64) and 512.
// Not faster: four softmax warpgroups, on one tile or in pairs on two; 8 warps
// for K; integer instead of converting dequantisation; rolled issue loops;
// rolled conversion loops.
//   warps  0.. 3  K tile: a token a thread, D/64 chunks of 32 elements
//   warps  4..11  V^T tile: a head_dim row a thread, D/64 pages
//   warps 12..15  softmax of the tile's keys  0..31: a query row a thread
//   warps 16..19  softmax of the tile's keys 32..63
//   warp  20      TMA: the tile's 4 page blocks into a 4-stage ring
//   warps 21, 22  issue the score and the value MMAs
// Warps 4..19 also bring Q in and write the output. Every wait is bounded; a
// timeout sets NVKV_DEVERR_TIMEOUT and drains.
//
// Measured, 24/4 heads, head_dim 256: the long prefill (65,536 + 2,048
// tokens, cap 50) 3.86 ms = 867 TFLOP/s, 0.52 of the measured matrix rate (3.95
// ms, 0.51, under steady load), bound by the softmax. A CTA of few tiles is bound by its way in and out,
// some 19,000 cycles for one tile: 3,100 to the tile's key range and the
// barriers, 2,800 to the first page block and Q, 4,000 for K and its scores,
// 2,400 for the first softmax, 3,600 for the output, 2,900 from its end to
// the next CTA's start on the SM. Packed documents of 1,500 tokens (8,192 +
// 2,048): 84.5 us = 481 TFLOP/s; windows of 1,024 in chunks of 512, 301, 777
// and 65 tokens: 81 us, 2.16 waves of such CTAs. A verify step of 24 rows
// over 2 x 32,768 tokens, 18 CTAs a pair: 46 us; its K and V^T warps are busy
// 2,000 of the 2,130 cycles a tile. (Reading a tile's bytes while the tile
// before is converted gained nothing there and cost the long prefill 11 %.)
#include <cfloat>
#include <type_traits>

#include "score_mod.cuh"
#include "sm100.cuh"

namespace nvkv {

bool make_pool_tmap(const nvkv_cache &c, CUtensorMap *map);

namespace {

using namespace sm100;

constexpr int kTileTokens = 64;
constexpr int kTilePages = 4;
constexpr int kStages = 4;
constexpr int kKWarps = 4;        // warps 0..3
constexpr int kVWarps = 8;        // warps 4..11
constexpr int kDeqWarps = kKWarps + kVWarps;
constexpr int kSmxWarps = 8;      // two warpgroups: warps 12..15 and 16..19
constexpr int kProducerWarp = 20;
constexpr int kMmaWarp = 21;      // issues the score MMAs
                                  // (warp 22 the value MMAs)
constexpr int kThreads = 23 * 32;
constexpr int kHalf = kTileTokens / 2;  // keys of a softmax thread
constexpr uint32_t kTmemCols = 512;
constexpr long long kWaitBudget = 2000000000LL;
constexpr float kLazyRescale = 8.0f;

// Tensor Memory columns (head_dim 128 uses half of Q's and O's).
constexpr uint32_t kColQ = 0;     // 128: Q (row lanes, d pairs)
constexpr uint32_t kColS = 128;   // 2 x 64: S slots (P overwrites the first 32 columns)
constexpr uint32_t kColO = 256;   // 256: O (row lanes, fp32 d)

// Sizes and shared memory. A page's kv-head block is staged as 128-byte rows
// with the 128-byte TMA swizzle: byte `off` of the block lies at swz(off).
template <int D>
struct Cfg {
  static_assert(D == 128 || D == 256, "head_dim");
  static constexpr int kHeadBytes = 18 * D;
  static constexpr int kRowsPerHead = kHeadBytes / 128;
  static constexpr int kPagePitch = (kHeadBytes + 1023) / 1024 * 1024;
  static constexpr int kStageBytes = kTilePages * kPagePitch;
  static constexpr int kKTileBytes = kTileTokens * D * 2;
  static constexpr int kVTileBytes = D * kTileTokens * 2;
  static constexpr int kOffK = kStages * kStageBytes;
  static constexpr int kOffV = kOffK + 2 * kKTileBytes;
  // V scales of a tile as f16 pairs [page][group][8], two tables (tile parity)
  static constexpr int kVscBytes = kTilePages * (D / 16) * 8 * 4;
  static constexpr int kOffVsc = kOffV + 2 * kVTileBytes;
  static constexpr int kOffRed = kOffVsc + 2 * kVscBytes;           // float[2][128]: a half's maxima
  static constexpr int kOffL = kOffRed + 2 * 128 * 4;               // float[2][128]: denominators
  static constexpr int kOffPages = kOffL + 2 * 128 * 4;             // int[stages][4]
  static constexpr int kOffPres = kOffPages + kStages * kTilePages * 4;  // u32[4]
  static constexpr int kOffFlags = kOffPres + 16;
  static constexpr int kOffSeen = kOffFlags + 16;                   // u64[stages]
  static constexpr int kOffBars = kOffSeen + kStages * 8;
  // full, empty; kready, vready, sready, pready, pvdone; qready, final, lready, final_qk
  static constexpr int kNumBars = 2 * kStages + 2 * 5 + 4;
  static constexpr int kOffTmem = kOffBars + kNumBars * 8;
  static constexpr int kSmemBytes = kOffTmem + 16 + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  static_assert(128 * (4 * D + 16) <= kOffVsc, "the output rows fit below the tables");
  static_assert(kOffK % 1024 == 0 && kOffPages % 16 == 0 && kOffSeen % 8 == 0 && kOffBars % 8 == 0, "alignment");
};

// Keeps what follows out of the way of the instructions that always run.
__device__ __forceinline__ bool rare(bool b) { return __builtin_expect(b, 0); }

__device__ __forceinline__ int swz(int off) { return off ^ ((off >> 3) & 0x70); }

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *flags,
                                         int32_t *err) {
  return guarded_wait(bar, parity, flags + 2, err, kWaitBudget);  // flags[2]: abort
}

__device__ __forceinline__ uint32_t dup_scale(uint32_t byte) {
  return e4m3x2_to_f16x2(byte | (byte << 8));
}

struct Args {
  int num_pages, Hkv;
  const int32_t *page_table;
  int max_pages;
  const int32_t *kv_lens;
  int max_kv_len;
  const __nv_bfloat16 *q;
  const int32_t *cu_q;
  int T;                 // > 0: a decode step of T queries per sequence (cu_q is not used,
                         // key_starts has one entry per sequence); 0: a chunk
  int total_q, Hq;
  float qscale;
  __nv_bfloat16 *out;
  int num_splits;
  float *ws_o, *ws_lse;  // null when num_splits is 1
  int32_t *err;
};

// kCopies = 4 or 2: tiles of at most 32 or 64 rows (a verify step, a decode
// step of a wide group, a short chunk).  The MMA has 128 rows anyway, so the
// rows stand in every (every other) 32-lane quarter of the tile, and each
// copy of a row weighs its own quarter (half) of every tile's keys, with a
// running maximum of its own and weights of 0 elsewhere; the copies are added
// at the end as key splits are.  The softmax of a tile then takes a quarter
// (half) of the instructions.
template <int D, int kCopies, class Mod>
__global__ void __launch_bounds__(kThreads, 1)
prefill_mod_kernel(const __grid_constant__ CUtensorMap tmap, const Args a, const Mod mod) {
  using C = Cfg<D>;
  constexpr int kTileRows = 128 / kCopies;
  constexpr int kQuarters = 4 / kCopies;    // 32-lane quarters of one copy
  constexpr int kKeys = kHalf / kCopies;    // keys of a softmax thread
  constexpr int kPagePitch = C::kPagePitch, kStageBytes = C::kStageBytes,
                kKTileBytes = C::kKTileBytes, kVTileBytes = C::kVTileBytes;
  // blockIdx.x = m-tile * num_splits + split: split s of an m-tile takes the
  // s-th of num_splits equal runs of its key tiles and, when num_splits > 1,
  // leaves O / l and log2(l) + m of its rows in the workspace for the merge.
  // The kernel before may still be running (programmatic dependent launch). The
  // merge in turn may be set up while this one runs, but not earlier: it reads
  // the chunk bounds ahead of its own wait.
  grid_dependency_wait();
  launch_dependents();
  const int mt = blockIdx.x / a.num_splits, split = blockIdx.x % a.num_splits;
  const int h = blockIdx.y, b = blockIdx.z;
  const int G = a.Hq / a.Hkv;
  const int q0 = a.T > 0 ? b * a.T : a.cu_q[b];
  const int n_b = a.T > 0 ? a.T : a.cu_q[b + 1] - q0;
  const int kv_len = a.kv_lens[b];
  auto start_of = [&](int i) { return mod.start(a.T > 0 ? b : q0 + i); };
  const int prefix = mod.prefix_of(b);
  const int rows = n_b * G;
  if (kTileRows * mt >= rows) return;  // uniform: this tile has no query row
  // (a decode step may have more queries than tokens: the first see nothing)
  const bool bad = n_b < 0 || q0 < 0 || q0 + n_b > a.total_q || (a.T == 0 && kv_len < n_b) ||
                   kv_len > a.max_kv_len || kv_len > a.max_pages * kPageTokens;
  // Output rows exist only when the chunk lies inside the total_q rows.
  const bool rows_ok = n_b >= 0 && q0 >= 0 && q0 + n_b <= a.total_q;

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint8_t *stages = smem;
  uint8_t *ktiles = smem + C::kOffK;
  uint8_t *vtiles = smem + C::kOffV;
  uint32_t *vsc = reinterpret_cast<uint32_t *>(smem + C::kOffVsc);  // [2][page][group][8]
  float *red_s = reinterpret_cast<float *>(smem + C::kOffRed);
  float *l_s = reinterpret_cast<float *>(smem + C::kOffL);
  int32_t *spages = reinterpret_cast<int32_t *>(smem + C::kOffPages);
  // Bit p of entry (tile & 3) is set when page p of the tile is present, so
  // the softmax leaves the keys of an absent page out. Written with the
  // tile's K; the K of tile j + 4 is written after the scores of tile j + 2,
  // which wait for the value MMAs of tile j.
  volatile uint32_t *present = reinterpret_cast<volatile uint32_t *>(smem + C::kOffPres);
  volatile int *flags = reinterpret_cast<volatile int *>(smem + C::kOffFlags);
  uint64_t *seen_s = reinterpret_cast<uint64_t *>(smem + C::kOffSeen);  // with gaps: keys seen
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBars);
  uint64_t *full = bars, *empty = bars + kStages;
  uint64_t *kready = bars + 2 * kStages, *vready = kready + 2, *sready = kready + 4,
           *pready = kready + 6, *pvdone = kready + 8, *qready = kready + 10,
           *final_bar = kready + 11, *lready = kready + 12, *final_qk = kready + 13;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffTmem);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (bad && threadIdx.x == 0) report(a.err, NVKV_DEVERR_LENGTH);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kDeqWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kready[i], kKWarps);
      mbar_init(&vready[i], kVWarps);
      mbar_init(&sready[i], 1);
      mbar_init(&pready[i], kSmxWarps);
      mbar_init(&pvdone[i], 1);
    }
    mbar_init(qready, 16);
    mbar_init(final_bar, 1);
    mbar_init(final_qk, 1);
    mbar_init(lready, kSmxWarps);
    fence_mbar_init();
  }
  if (threadIdx.x < 4) flags[threadIdx.x] = 0;
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }

  // The query rows, asked for before anything else is worked out: coalesced
  // copies into the second K and V tile slots (free until the second tile),
  // 16-byte chunks swizzled so that a row a lane reads them without bank
  // conflicts. (Each lane loading its own row took 4,000 cycles of the
  // load unit, and the page ids queued behind it.)
  auto q_chunk = [&](int rr, int c) -> uint8_t * {
    return (rr < 64 ? ktiles + kKTileBytes : vtiles + kVTileBytes) + (rr & 63) * (D * 2) +
           ((c ^ (rr & 7)) << 4);
  };
  if (warp >= kKWarps && warp < kProducerWarp) {
    constexpr int kRowChunks = D / 8, kAtOnce = 32 / kRowChunks;  // rows of an instruction
    constexpr int kWarpRows = kTileRows / 16;
    const int r0 = (warp - kKWarps) * kWarpRows, c = lane % kRowChunks;
    // lane i knows where the warp's row i is (a division once)
    const int mine = kTileRows * mt + r0 + lane % kWarpRows;
    const int at = mine < rows && !bad ? mine / G * a.Hq + mine % G : -1;
#pragma unroll
    for (int i = 0; i < kWarpRows; i += kAtOnce) {
      const int rr = i + lane / kRowChunks, from = __shfl_sync(0xffffffffu, at, rr);
      uint8_t *dst = q_chunk(r0 + rr, c);
      if (from >= 0)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)),
                     "l"(a.q + ((size_t)q0 * a.Hq + h * G + from) * D + 8 * c)
                     : "memory");
      else
        *reinterpret_cast<uint4 *>(dst) = make_uint4(0u, 0u, 0u, 0u);
    }
  }

  // The keys from key_lo to key_hi - 1 hold all that any row of the tile sees:
  // every warp scans the tile's tokens. Rows with starts of their own may
  // leave keys unseen in between (padding between documents sees nothing):
  // there are none when each row's interval touches the next one's. (Without
  // starts, and in a decode step, it does: all that see a key see their own
  // position, or the step's first key.)
  int key_lo = 0x7fffffff, key_hi = 0;
  bool gaps = false;
  const int i_first = kTileRows * mt / G;
  const int i_last = min(n_b - 1, (kTileRows * mt + kTileRows - 1) / G);
  auto range_of = [&](int i, int &lo, int &hi) {
    key_range(kv_len - n_b + i, kv_len, start_of(i), mod.window, prefix, lo, hi);
  };
  if (!bad) {
    for (int i = i_first + lane; i <= i_last; i += 32) {
      int lo, hi;
      range_of(i, lo, hi);
      if (lo < hi) key_lo = min(key_lo, lo), key_hi = max(key_hi, hi);
      if (mod.starts && a.T == 0 && i < i_last) {
        int lo2, hi2;
        range_of(i + 1, lo2, hi2);
        gaps |= lo >= hi || lo2 >= hi2 || lo > hi2 || lo2 > hi;
      }
    }
  }
  gaps = __any_sync(0xffffffffu, gaps);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    key_lo = min(key_lo, __shfl_xor_sync(0xffffffffu, key_lo, o));
    key_hi = max(key_hi, __shfl_xor_sync(0xffffffffu, key_hi, o));
  }
  if (key_lo >= key_hi) key_lo = key_hi = 0;  // nothing is seen
  const int tile_lo = key_lo / kTileTokens;
  const int ntiles_all = (key_hi + kTileTokens - 1) / kTileTokens - tile_lo;
  // This CTA's key tiles j0 .. j0 + ntiles - 1, with a bias counted from the
  // newest; every ring and barrier below counts from its first tile.
  const int j0 = (int)((int64_t)split * ntiles_all / a.num_splits);
  const int ntiles = (int)((int64_t)(split + 1) * ntiles_all / a.num_splits) - j0;
  auto tile_key = [&](int j) {
    return (tile_lo + (Mod::kBias ? ntiles_all - 1 - (j0 + j) : j0 + j)) * kTileTokens;
  };

  // (the TMA warp) which of tile j's 64 keys some row sees, where there may be
  // gaps; a row of the tile at a time in every lane
  auto seen_keys = [&](int j) -> uint64_t {
    if (!gaps) return ~uint64_t(0);
    const int tok = tile_key(j);
    uint64_t seen = 0;
    for (int i = i_first + lane; i <= i_last; i += 32) {
      int lo, hi;
      range_of(i, lo, hi);
      lo = max(lo - tok, 0), hi = min(hi - tok, kTileTokens);
      if (lo < hi) seen |= (~uint64_t(0) << lo) & (~uint64_t(0) >> (kTileTokens - hi));
    }
    return (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(seen >> 32)) << 32 |
           __reduce_or_sync(0xffffffffu, (uint32_t)seen);
  };
  // pages of the tiles: lane p's of every four
  const int32_t *pt = a.page_table + (size_t)b * a.max_pages;
  const int p = lane & 3;
  auto page_for = [&](int j, uint64_t seen) -> int {
    const int tok = tile_key(j) + p * kPageTokens;
    if (tok >= key_hi || tok + kPageTokens <= key_lo) return -1;  // nobody sees it
    if (((seen >> (kPageTokens * p)) & 0xffffu) == 0) return -1;
    const int pg = pt[tok / kPageTokens];
    if (pg < 0 || pg >= a.num_pages) {
      if (lane < kTilePages) report(a.err, NVKV_DEVERR_PAGE_ID);
      return -1;
    }
    return pg;
  };
  int first_page = -1;
  uint64_t first_seen = 0;
  if (warp == kProducerWarp) {
    prefetch_tmap(&tmap);
    if (ntiles > 0) first_page = page_for(0, first_seen = seen_keys(0));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  float qfac = 1.f;  // a softmax thread's row: what its products become scores by
  if (warp >= kKWarps && warp < kProducerWarp) {
    // Q row -> Tensor Memory (A operand), f16: lane quarter warp % 4, a quarter
    // of the columns each.
    const int lq = warp & 3, part = (warp - kKWarps) >> 2;
    const int rr = 32 * (lq % kQuarters) + lane;
    asm volatile("cp.async.wait_all;" ::: "memory");
    named_barrier(10, 16 * 32);  // every warp's rows are there
    uint32_t qw[D / 8], top2 = 0;
#pragma unroll
    for (int v = 0; v < D / 32; ++v) {
      const uint4 r4 = *reinterpret_cast<const uint4 *>(q_chunk(rr, part * (D / 32) + v));
      qw[4 * v] = r4.x, qw[4 * v + 1] = r4.y, qw[4 * v + 2] = r4.z, qw[4 * v + 3] = r4.w;
    }
#pragma unroll
    for (int v = 0; v < D / 8; ++v) top2 = __vmaxu2(top2, qw[v] & 0x7fff7fffu);
    // the row's largest exponent, from the four quarters' maxima (where the
    // softmax keeps its maxima and denominators later)
    static_assert(C::kOffL == C::kOffRed + 2 * 128 * 4, "one table");
    uint32_t *top_s = reinterpret_cast<uint32_t *>(red_s) + 32 * lq + lane;  // [part][row]
    top_s[128 * part] = max(top2 >> 16, top2 & 0xffffu);
    named_barrier(10, 16 * 32);
    // (below 2^-100 a row's scores are below 2^-80 whatever the keys)
    const uint32_t eb = max(27u, max(max(top_s[0], top_s[128]), max(top_s[256], top_s[384])) >> 7);
    // 2^(14 - e), e = eb - 127, with the scale's sign, so that the factor is
    // positive; a row that is not finite is NaN throughout
    float up = a.qscale == 0.f ? 0.f : copysignf(__uint_as_float((268u - eb) << 23), a.qscale);
    if (eb == 255u) up = NAN;
    qfac = fmaxf(fabsf(a.qscale) * __uint_as_float((eb - 14u) << 23), FLT_MIN);  // 2^(e - 14)
#pragma unroll
    for (int c16 = 0; c16 < D / 128; ++c16) {
      uint32_t w[16];
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const uint32_t rw = qw[16 * c16 + v];
        const __half2 hh = __floats2half2_rn(__uint_as_float(rw << 16) * up,
                                             __uint_as_float(rw & 0xffff0000u) * up);
        w[v] = *reinterpret_cast<const uint32_t *>(&hh);
      }
      tmem_st16(tmem + ((uint32_t)(32 * lq) << 16) + kColQ + part * (D / 8) + c16 * 16, w);
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(qready);
  }

  if (warp >= kProducerWarp) {
    if (warp == kProducerWarp) {
      // ---------------------------------------------------------------- TMA
      int cur = first_page;
      uint64_t cur_seen = first_seen;
      for (int j = 0; j < ntiles; ++j) {
        const int stage = j % kStages;
        const uint64_t nxt_seen = j + 1 < ntiles ? seen_keys(j + 1) : 0;
        const int nxt = j + 1 < ntiles ? page_for(j + 1, nxt_seen) : -1;
        if (j >= kStages) {
          if (lane == 0) wait_bar(&empty[stage], ((j / kStages) + 1) & 1, flags, a.err);
          __syncwarp();
        }
        const bool mine = lane < kTilePages && cur >= 0;
        if (lane < kTilePages) spages[stage * kTilePages + lane] = cur;
        if (lane == 0) seen_s[stage] = cur_seen;
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * C::kHeadBytes;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], bytes);
        __syncwarp();
        if (mine)
          tma_load_2d(stages + stage * kStageBytes + lane * kPagePitch, &tmap, 0,
                      (cur * a.Hkv + h) * C::kRowsPerHead, &full[stage]);
        cur = nxt, cur_seen = nxt_seen;
      }
      // Drain: every issued copy must land before the CTA may exit.
      if (lane == 0) {
        const int first = ntiles > kStages ? ntiles - kStages : 0;
        for (int k = first; k < ntiles; ++k)
          mbar_wait(&full[k % kStages], (k / kStages) & 1, kWaitBudget);
      }
      __syncwarp();
    } else if (ntiles > 0) {
      // ---------------------------------------------------------------- MMA
      // Two issuing warps: issuing a batch of tcgen05.mma blocks the thread
      // until it has nearly executed, so a single one held the value MMAs of
      // a tile back behind the next tile's scores, and with them the S slot
      // that the scores after those wait for. The whole warp walks the loop
      // and one lane issues (see mma_f16_ts_warp).
      const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
      const int nt = (int)__reduce_max_sync(0xffffffffu, (uint32_t)ntiles);
      auto aborted = [&]() { return __any_sync(0xffffffffu, flags[2]); };
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        wait_bar(bar, parity, flags, a.err);
        __syncwarp();
      };
      bool issued = false;
      if (warp == kMmaWarp) {
        const uint32_t idesc_qk = idesc_f16_f32(128, kTileTokens, false, false);
        const uint32_t kb = smem_u32(ktiles);
        wait(qready, 0);
        for (int j = 0; j < nt && !aborted(); ++j) {
          const int slot = j & 1;
          wait(&kready[slot], (j >> 1) & 1);
          // the S slot: P of tile j-2 there has been used
          if (j >= 2) wait(&pvdone[slot], ((j >> 1) + 1) & 1);
          tc_fence_after();
          const uint64_t kd = smem_desc(kb + slot * kKTileBytes, 1024, 128);
          const uint32_t scol = tm + kColS + slot * 64;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_f16_ts_warp(scol, tm + kColQ + ks * 8, desc_at(kd, ks * 2 * 1024), idesc_qk, ks > 0);
          mma_commit_warp(&sready[slot]);
          issued = true;
        }
        if (issued) {
          mma_commit_warp(final_qk);
          mbar_wait(final_qk, 0, kWaitBudget);
        }
      } else {
        const uint32_t idesc_pv = idesc_f16_f32(128, D, false, false);
        const uint32_t vb = smem_u32(vtiles);
        for (int j = 0; j < nt && !aborted(); ++j) {
          const int slot = j & 1;
          wait(&vready[slot], (j >> 1) & 1);
          wait(&pready[slot], (j >> 1) & 1);
          tc_fence_after();
          const uint32_t pcol = tm + kColS + slot * 64;  // P: first 32 columns of the slot
          const uint64_t vd = smem_desc(vb + slot * kVTileBytes, D * 16, 128);
#pragma unroll
          for (int ks = 0; ks < kTileTokens / 16; ++ks)
            mma_f16_ts_warp(tm + kColO, pcol + ks * 8, desc_at(vd, ks * 2 * (D * 16)), idesc_pv,
                            j > 0 || ks > 0);
          mma_commit_warp(&pvdone[slot]);
          issued = true;
        }
        if (issued) {
          mma_commit_warp(final_bar);
          mbar_wait(final_bar, 0, kWaitBudget);
        }
      }
      __syncwarp();
    }
  } else if (warp < kDeqWarps) {
    if (warp < kKWarps) {
      // ------------------------------------------------------------------ K
      const int t = threadIdx.x;  // 0..127
      constexpr int kChunks = D / 64;
      // thread = token n (32 consecutive per warp), chunks kChunks * cp + ..
      const int n = t & 63, cp = t >> 6;
      const int p = n >> 4, s = n & 15;
      for (int j = 0; j < ntiles; ++j) {
        const int stage = j % kStages, slot = j & 1;
        const uint8_t *pg = stages + stage * kStageBytes + p * kPagePitch;
        wait_bar(&full[stage], (j / kStages) & 1, flags, a.err);
        const int4 pgs = *reinterpret_cast<const int4 *>(spages + stage * kTilePages);
        const int tok = tile_key(j) + n;
        const int mine = p < 2 ? (p == 0 ? pgs.x : pgs.y) : (p == 2 ? pgs.z : pgs.w);
        const bool ok = mine >= 0 && tok >= key_lo && tok < key_hi;
        // The stage's bytes, before the wait for the tile slot.
        uint4 w4[kChunks];
        uint2 sc = make_uint2(0u, 0u);  // scale bytes of the chunks' groups (two a chunk)
#pragma unroll
        for (int ci = 0; ci < kChunks; ++ci) w4[ci] = make_uint4(0u, 0u, 0u, 0u);
        if (ok) {
          const uint8_t *sp = pg + swz(ks_off(D) + s * (D / 16) + 2 * kChunks * cp);
          if constexpr (kChunks == 4)
            sc = *reinterpret_cast<const uint2 *>(sp);
          else
            sc.x = *reinterpret_cast<const uint32_t *>(sp);
#pragma unroll
          for (int ci = 0; ci < kChunks; ++ci)
            w4[ci] = *reinterpret_cast<const uint4 *>(
                pg + swz(s * (D / 2) + (kChunks * cp + ci) * 16));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);  // this warp's reads of the stage are done
        // K tile slot: its previous tile's scores must be done (the second
        // slot holds Q at first).
        if (j == 1) wait_bar(qready, 0, flags, a.err);
        if (j >= 2) {
          wait_bar(&sready[slot], ((j >> 1) + 1) & 1, flags, a.err);
          tc_fence_after();
        }
        if (t == 0)
          present[j & 3] = (pgs.x >= 0 ? 1u : 0u) | (pgs.y >= 0 ? 2u : 0u) |
                           (pgs.z >= 0 ? 4u : 0u) | (pgs.w >= 0 ? 8u : 0u);
        uint8_t *kt = ktiles + slot * kKTileBytes + (n >> 3) * 128 + (n & 7) * 16;
#pragma unroll
        for (int ci = 0; ci < kChunks; ++ci) {
          const int c = kChunks * cp + ci;  // 32-d chunk: groups 2c, 2c+1
          const uint32_t two = (ci < 2 ? sc.x : sc.y) >> (16 * (ci & 1));
          const uint32_t s0 = dup_scale(two & 0xffu), s1 = dup_scale((two >> 8) & 0xffu);
          const uint32_t w[4] = {w4[ci].x, w4[ci].y, w4[ci].z, w4[ci].w};
          // K-major core matrices: element (n, k) at (k/8)*1024 + (n/8)*128 + (n%8)*16.
#pragma unroll
          for (int wi = 0; wi < 4; ++wi) {
            uint32_t t4[4];
            e2m1x8_to_f16x2x4(w[wi], t4);
            const uint32_t s2 = wi < 2 ? s0 : s1;
            *reinterpret_cast<uint4 *>(kt + (4 * c + wi) * 1024) =
                make_uint4(hmul2_u32(t4[0], s2), hmul2_u32(t4[1], s2), hmul2_u32(t4[2], s2),
                           hmul2_u32(t4[3], s2));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kready[slot]);
      }
    } else {
      // ------------------------------------------------------------------ V
      const int t = threadIdx.x - kKWarps * 32;  // 0..255
      // thread = head_dim row d, pages p0 .. p0 + kPages - 1 of the tile
      constexpr int kPages = D / 64;
      const int d = t % D, p0 = D == 256 ? 0 : t / D * kPages;
      const int g = d >> 4;
      for (int j = 0; j < ntiles; ++j) {
        const int stage = j % kStages, slot = j & 1;
        const uint8_t *stg = stages + stage * kStageBytes;
        wait_bar(&full[stage], (j / kStages) & 1, flags, a.err);
        const int4 pg4 = *reinterpret_cast<const int4 *>(spages + stage * kTilePages);
        const uint64_t seen = seen_s[stage];
        const int tok0 = tile_key(j);
        if (t < D) {
          // This tile's V scales, converted once (the 16 V^T rows of a group
          // share them): a thread takes 4 consecutive tokens of one (page,
          // group). (Absent pages convert stale bytes that are never used.)
          const int p = t / (D / 4), gg = (t >> 2) % (D / 16), q4 = t & 3;
          const uint32_t raw = *reinterpret_cast<const uint32_t *>(
              stg + p * kPagePitch + swz(vs_off(D) + gg * kPageTokens) + 4 * q4);
          uint32_t t2[2];
          e4m3x4_to_f16x2x2(raw, t2);
          *reinterpret_cast<uint2 *>(vsc + ((slot * kTilePages + p) * (D / 16) + gg) * 8 + 2 * q4) =
              make_uint2(t2[0], t2[1]);
        }
        uint2 cw[kPages];
#pragma unroll
        for (int pp = 0; pp < kPages; ++pp)
          cw[pp] = *reinterpret_cast<const uint2 *>(stg + (p0 + pp) * kPagePitch +
                                                    swz(vc_off(D) + d * 8));
        // The scale table of this tile is complete once every V thread is
        // here; all of them finished reading the table of tile j-2 before
        // arriving here for tile j-1.
        named_barrier(1, kVWarps * 32);
        if (lane == 0) mbar_arrive(&empty[stage]);  // (the barrier follows every read)
        // V^T tile slot: its previous tile's value MMAs must be done.
        if (j == 1) wait_bar(qready, 0, flags, a.err);
        if (j >= 2) {
          wait_bar(&pvdone[slot], ((j >> 1) + 1) & 1, flags, a.err);
          tc_fence_after();
        }
        uint8_t *vt = vtiles + slot * kVTileBytes + (d >> 3) * 128 + (d & 7) * 16;
#pragma unroll
        for (int pp = 0; pp < kPages; ++pp) {
          const int p = p0 + pp;
          const int ptok = tok0 + p * kPageTokens;
          const int mine = p == 0 ? pg4.x : p == 1 ? pg4.y : p == 2 ? pg4.z : pg4.w;
          uint32_t o8[8];
          if (!rare(mine < 0)) {
            const uint4 *tb = reinterpret_cast<const uint4 *>(
                vsc + ((slot * kTilePages + p) * (D / 16) + g) * 8);
            const uint4 sa = tb[0], sb = tb[1];
            const uint32_t sp[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
            uint32_t c0[4], c1[4];
            e2m1x8_to_f16x2x4(cw[pp].x, c0);
            e2m1x8_to_f16x2x4(cw[pp].y, c1);
#pragma unroll
            for (int e = 0; e < 8; ++e) o8[e] = hmul2_u32(e < 4 ? c0[e] : c1[e - 4], sp[e]);
            if (rare(gaps || ptok < key_lo || ptok + kPageTokens > key_hi)) {
              // tokens that no row sees are zero, whatever their bytes
              const uint32_t some = (uint32_t)(seen >> (kPageTokens * p));
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int t0 = ptok + 2 * e;
                if (t0 < key_lo || t0 >= key_hi || !((some >> (2 * e)) & 1u)) o8[e] &= 0xffff0000u;
                if (t0 + 1 < key_lo || t0 + 1 >= key_hi || !((some >> (2 * e + 1)) & 1u))
                  o8[e] &= 0xffffu;
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) o8[e] = 0u;
          }
          // K-major (tokens) core matrices: element (d, t) at (t/8)*16*D + (d/8)*128 + (d%8)*16.
          *reinterpret_cast<uint4 *>(vt + (2 * p) * (16 * D)) =
              make_uint4(o8[0], o8[1], o8[2], o8[3]);
          *reinterpret_cast<uint4 *>(vt + (2 * p + 1) * (16 * D)) =
              make_uint4(o8[4], o8[5], o8[6], o8[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&vready[slot]);
      }
    }
  } else {
    // ------------------------------------------------------------- softmax
    const int hf = warp >= kDeqWarps + 4;     // keys 32 * hf .. of every tile
    const int lq = warp & 3;
    const int copy = lq / kQuarters;
    const int koff = kHalf * hf + kKeys * copy;  // first key of this thread in a tile
    const int r = 32 * lq + lane;             // row of the MMA
    const uint32_t tl = tmem + ((uint32_t)(32 * lq) << 16);
    const int gr = kTileRows * mt + 32 * (lq % kQuarters) + lane;
    const bool valid = gr < rows && !bad;
    const int i = gr / G, g = gr % G;
    const int pos = kv_len - n_b + i;
    int row_lo = 0, row_hi = 0;               // keys row_lo .. row_hi - 1 are visible
    float slope2 = 0.f;
    if (valid) {
      key_range(pos, kv_len, start_of(i), mod.window, prefix, row_lo, row_hi);
      slope2 = mod.slope2(h * G + g);
    }
    // (a row that is none has scores of 0 and a maximum of 0: it never asks
    // for a new one)
    float m = valid ? -INFINITY : 0.f, l = 0.f;
    // Scores that are neither capped nor biased stay products: one multiply-add
    // brings in the factor and subtracts the maximum. (Documents 86.0 -> 84.5
    // us.) The maximum is a rounded product, so all of a row's weights are off
    // by the same power of two, up to half of the maximum's last place: past
    // kRawMost, where that could leave f16 (2^8 by the lag, 2^4 by the roundings
    // at most), the tile's products become scores first.
    constexpr bool kRaw = !Mod::kCap && !Mod::kBias;
    constexpr float kRawMost = 33554432.f;  // 2^25
    for (int j = 0; j < ntiles; ++j) {
      const int slot = j & 1;
      wait_bar(&sready[slot], (j >> 1) & 1, flags, a.err);
      __syncwarp();  // the Tensor Memory loads below are warp-collective
      tc_fence_after();
      const uint32_t scol = tl + kColS + slot * 64;
      float x[kKeys];
      auto to_scores = [&]() {
#pragma unroll
        for (int e = 0; e < kKeys; e += 2) {
          const float2 v = mul_f32x2(make_float2(x[e], x[e + 1]), make_float2(qfac, qfac));
          x[e] = v.x, x[e + 1] = v.y;
        }
      };
      auto load_scores = [&]() {
        uint32_t(&xr)[kKeys] = reinterpret_cast<uint32_t(&)[kKeys]>(x);
        if constexpr (kKeys == 8) {
          tmem_ld8(scol + koff, xr);
        } else {
#pragma unroll
          for (int e = 0; e < kKeys; e += 16)
            tmem_ld16(scol + koff + e, reinterpret_cast<uint32_t(&)[16]>(xr[e]));
        }
        tmem_wait_ld();
        if constexpr (!kRaw) to_scores();
      };
      auto top_score = [&]() {
        float t0 = max3(x[0], x[1], x[2]), t1 = max3(x[3], x[4], x[5]);
#pragma unroll
        for (int e = 6; e + 4 <= kKeys; e += 4) {
          t0 = max3(t0, x[e], x[e + 1]);
          t1 = max3(t1, x[e + 2], x[e + 3]);
        }
        const float top = max3(t0, t1, fmaxf(x[kKeys - 2], x[kKeys - 1]));
        return kRaw ? top * qfac : top;
      };
      load_scores();
      const int key0 = tile_key(j) + koff;
      float above;  // no visible score is larger
      if constexpr (Mod::kCap) {
        // A polynomial, good for scores of at most 0.75 caps and increasing
        // beyond: its own values tell whether all of them are. Where one is
        // not, the exact form (two special functions a score).
#pragma unroll
        for (int e = 0; e < kKeys; e += 2) {
          const float2 v = cap_small(mod, make_float2(x[e], x[e + 1]));
          x[e] = v.x, x[e + 1] = v.y;
        }
        float t0 = max3_abs(x[0], x[1], x[2]), t1 = max3_abs(x[3], x[4], x[5]);
#pragma unroll
        for (int e = 6; e + 4 <= kKeys; e += 4) {
          t0 = max3_abs(t0, x[e], x[e + 1]);
          t1 = max3_abs(t1, x[e + 2], x[e + 3]);
        }
        above = max3_abs(t0, t1, max3_abs(x[kKeys - 2], x[kKeys - 1], 0.f));
        if (rare(__any_sync(0xffffffffu, !(above <= mod.cap_top)))) {  // (a NaN too)
          load_scores();
#pragma unroll
          for (int e = 0; e < kKeys; e += 2) {
            const float2 v = mod.cap(make_float2(x[e], x[e + 1]));
            x[e] = v.x, x[e + 1] = v.y;
          }
          above = mod.cap2;
        }
      } else {
        above = top_score();
      }
      if constexpr (Mod::kBias) {
        // (distances are exact; with a prefix a key may lie ahead)
        const float d0 = (float)(pos - key0);
#pragma unroll
        for (int e = 0; e < kKeys; ++e) x[e] = fmaf(-slope2, fabsf(d0 - (float)e), x[e]);
        above = top_score();
      }
      if (rare(key0 < row_lo || key0 + kKeys > row_hi)) {
#pragma unroll
        for (int e = 0; e < kKeys; ++e)
          if (key0 + e < row_lo || key0 + e >= row_hi) x[e] = -INFINITY;
        if (valid && (key0 >= row_hi || key0 + kKeys <= row_lo)) above = -INFINITY;
      }
      const uint32_t here = present[j & 3] >> (koff / kPageTokens);
      constexpr uint32_t kHere = kKeys > kPageTokens ? 3u : 1u;  // their pages
      if (rare((here & kHere) != kHere)) {
#pragma unroll
        for (int e = 0; e < kKeys; ++e)
          if (!((here >> (e / kPageTokens)) & 1u)) x[e] = -INFINITY;
      }
      // One barrier of the two warps that share these rows: may any score
      // pass its row's running maximum by 2^8? (Every score of the tile has
      // been read once it is passed.) The difference is exact where it matters;
      // m + 8 is not past 2^27, where its rounding let a weight of 2^16 pass.
      if (rare(named_barrier_or(2 + lq, 64, above - m > kLazyRescale))) {
        // The exact maximum of the row's visible scores decides; both threads
        // of the row come to the same result.
        red_s[128 * hf + r] = top_score();
        named_barrier(2 + lq, 64);
        const float tmax = fmaxf(red_s[r], red_s[128 + r]);
        const bool raise = tmax > -INFINITY && (m == -INFINITY || tmax - m > kLazyRescale);
        const float alpha = raise ? exp2f(m - tmax) : 1.f;  // 0 when m = -inf
        // The Tensor Memory loads and stores of O are warp-collective: if any
        // row of the warp moves, the whole warp rescales its half of the
        // columns, rows that stay with alpha 1 -- once the value MMAs up to
        // tile j-1 are done.
        if (j > 0 && __any_sync(0xffffffffu, raise)) {
          wait_bar(&pvdone[(j - 1) & 1], ((j - 1) >> 1) & 1, flags, a.err);
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int c16 = 0; c16 < D / 32; ++c16) {
            uint32_t rr[16];
            const uint32_t col = tl + kColO + hf * (D / 2) + c16 * 16;
            tmem_ld16(col, rr);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
            tmem_st16(col, rr);
          }
          tmem_wait_st();
        }
        if (raise) {
          l *= alpha;
          m = tmax;
        }
        named_barrier(2 + lq, 64);  // the maxima have been read
      }
      // Weights from an fp32 exponential (as fast here as the f16 pair form,
      // whose results have to be widened again for the sum), rounded to f16
      // for the value MMAs; masked keys are -inf and give 0 (a row with no
      // visible key yet keeps m = -inf: it subtracts 0 instead). The
      // denominator sums the weights before their rounding, in fp32.
      const float ms = m == -INFINITY ? 0.f : m;
      float fac = kRaw ? qfac : 1.f;
      if (kRaw && rare(__any_sync(0xffffffffu, fabsf(ms) > kRawMost))) {
        to_scores();
        fac = 1.f;
      }
      uint32_t pw[kKeys / 2];
      float2 lv0 = make_float2(0.f, 0.f), lv1 = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < kKeys / 2; ++e) {
        const float2 two = make_float2(x[2 * e], x[2 * e + 1]), neg = make_float2(-ms, -ms);
        const float2 d = kRaw ? fma_f32x2(two, make_float2(fac, fac), neg) : add_f32x2(two, neg);
        float2 w;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w.x) : "f"(d.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w.y) : "f"(d.y));
        asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(pw[e]) : "f"(w.x), "f"(w.y));
        (e & 1 ? lv1 : lv0) = add_f32x2(e & 1 ? lv1 : lv0, w);
      }
      l += (lv0.x + lv0.y) + (lv1.x + lv1.y);
      // P overwrites the first 32 columns of its own S slot.
      if constexpr (kCopies == 1) {
        tmem_st16(scol + kHalf / 2 * hf, pw);
      } else {
        uint32_t all[kHalf / 2];
#pragma unroll
        for (int e = 0; e < kHalf / 2; ++e)
          all[e] = e / (kKeys / 2) == copy ? pw[e % (kKeys / 2)] : 0u;
        tmem_st16(scol + kHalf / 2 * hf, all);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pready[slot]);
    }
    l_s[128 * hf + r] = l;
    // (the maxima of the last tile that asked for one have been read)
    if (kCopies > 1 && hf == 0) red_s[r] = m;
    __syncwarp();
    if (lane == 0) mbar_arrive(lready);
    // Split partial: O / l (fp32) and lse = m + log2(l), -inf without a
    // visible key, in the split's plane of total_q * Hq rows.
    if (kCopies == 1 && a.ws_o && hf == 0) {
      wait_bar(lready, 0, flags, a.err);
      const float both = l_s[r] + l_s[128 + r];
      if (gr < rows && rows_ok)
        a.ws_lse[(size_t)split * a.total_q * a.Hq + (size_t)(q0 + i) * a.Hq + h * G + g] =
            both == 0.f ? -INFINITY : m + log2f(both);  // (NaN stays NaN)
    }
  }

  if (warp >= kKWarps && warp < kProducerWarp) {
    // ------------------------------------------------------------- epilogue
    // O / l -> out (or the split's plane), 16 warps: lane quarter warp % 4,
    // quarter warp / 4 of the columns.
    // lane i knows where row 32 * lq + i goes (-1: nowhere)
    int at = -1;
    if (kCopies == 1) {
      const int mine = 128 * mt + 32 * (warp & 3) + lane;
      if (mine < rows && rows_ok) at = mine / G * a.Hq + mine % G;
    }
    if (ntiles > 0) {
      wait_bar(final_bar, 0, flags, a.err);
      __syncwarp();
      tc_fence_after();
    }
    wait_bar(lready, 0, flags, a.err);
    const int lq = warp & 3, part = (warp - kKWarps) >> 2;
    const int r = 32 * lq + lane;
    const size_t plane = (size_t)split * a.total_q * a.Hq;
    auto out_row = [&](int gr) { return (size_t)(q0 + gr / G) * a.Hq + h * G + gr % G; };
    float inv;  // times O: 1 / l, with copies their share 2^(m - max) / sum 2^(m - max) l
    if constexpr (kCopies == 1) {
      const float l = l_s[r] + l_s[128 + r];
      inv = l > 0.f ? 1.f / l : 0.f;
    } else {
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int c = 0; c < kCopies; ++c) top = fmaxf(top, red_s[32 * (lq % kQuarters + kQuarters * c) + lane]);
      if (top == -INFINITY) top = 0.f;  // (no key seen)
#pragma unroll
      for (int c = 0; c < kCopies; ++c) {
        const int rc = 32 * (lq % kQuarters + kQuarters * c) + lane;
        sum = fmaf(exp2f(red_s[rc] - top), l_s[rc] + l_s[128 + rc], sum);
      }
      inv = sum > 0.f ? exp2f(red_s[r] - top) / sum : 0.f;
      const int gr = kTileRows * mt + 32 * lq + lane;
      if (a.ws_o && lq < kQuarters && part == 0 && gr < rows && rows_ok)
        a.ws_lse[plane + out_row(gr)] = sum == 0.f ? -INFINITY : top + log2f(sum);
    }
    const uint32_t tl = tmem + ((uint32_t)(32 * lq) << 16) + kColO + part * (D / 4);
    // The rows go through shared memory (nothing else uses it any more), 16
    // bytes apart from a multiple of 128 so that the lanes' stores meet no
    // bank conflict, and leave coalesced.
    const bool wide = kCopies > 1 || a.ws_o;
    const int bytes = wide ? D * 4 : D * 2;
    uint8_t *srow = smem + r * (bytes + 16);
#pragma unroll 1
    for (int c16 = 0; c16 < D / 64; ++c16) {
      uint32_t rr[16];
      if (ntiles > 0) {
        __syncwarp();
        tmem_ld16(tl + c16 * 16, rr);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) rr[e] = 0u;
      }
      const int col = part * (D / 4) + c16 * 16;
      if (wide) {
        float4 *dst = reinterpret_cast<float4 *>(srow + 4 * col);
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4)
          dst[e4] = make_float4(__uint_as_float(rr[4 * e4]) * inv,
                                __uint_as_float(rr[4 * e4 + 1]) * inv,
                                __uint_as_float(rr[4 * e4 + 2]) * inv,
                                __uint_as_float(rr[4 * e4 + 3]) * inv);
      } else {
        uint32_t ow[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(rr[2 * e]) * inv,
                                                    __uint_as_float(rr[2 * e + 1]) * inv);
          ow[e] = *reinterpret_cast<uint32_t *>(&b2);
        }
        uint4 *dst = reinterpret_cast<uint4 *>(srow + 2 * col);
        dst[0] = make_uint4(ow[0], ow[1], ow[2], ow[3]);
        dst[1] = make_uint4(ow[4], ow[5], ow[6], ow[7]);
      }
    }
    if constexpr (kCopies > 1) {
      // The copies' shares of a row added in order, a warp a row.
      named_barrier(10, 16 * 32);
      for (int rr = warp - kKWarps; rr < kTileRows; rr += 16) {
        const int gr = kTileRows * mt + rr;
        if (gr >= rows || !rows_ok) break;  // warp-uniform
        const size_t orow = out_row(gr);
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 128) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int c = 0; c < kCopies; ++c) {
            const float4 o = *reinterpret_cast<const float4 *>(
                smem + (rr + kTileRows * c) * (bytes + 16) + 4 * c0 + 16 * lane);
            v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
          }
          const size_t at = orow * D + c0 + 4 * lane;
          if (a.ws_o) {
            *reinterpret_cast<float4 *>(a.ws_o + plane * D + at) = v;
          } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
            *reinterpret_cast<uint2 *>(a.out + at) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
          }
        }
      }
    } else {
      named_barrier(6 + lq, 128);  // the four warps of these rows
      // Eight rows a warp, 16 bytes a lane.
      const int shift = __ffs(bytes / 16) - 1;  // (row bytes are a power of two)
      const size_t row0 = (size_t)q0 * a.Hq + h * G;
      uint8_t *first = a.ws_o ? (uint8_t *)(a.ws_o + (plane + row0) * D)
                              : (uint8_t *)(a.out + row0 * D);
#pragma unroll 4
      for (int k = lane; k < 8 << shift; k += 32) {
        const int i = 8 * part + (k >> shift), off = (k & ((1 << shift) - 1)) * 16;
        const int to = __shfl_sync(0xffffffffu, at, i);
        if (to >= 0)
          *reinterpret_cast<uint4 *>(first + (size_t)to * bytes + off) =
              *reinterpret_cast<const uint4 *>(smem + (32 * lq + i) * (bytes + 16) + off);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// Merge of the key splits: row (token, head) of `rows` is
// sum_s 2^(lse_s - M) O_s / sum_s 2^(lse_s - M) with M the largest lse (zero
// when no split saw a key). kW warps a row (a decode step's few rows have up
// to 32 splits), D/32 elements a lane; the warps' sums are added in order.
// A split whose lse is NaN makes the row NaN. Rows outside every sequence's
// chunk are left alone. Set up while the
// attention kernel runs (programmatic dependent launch).
constexpr int kMaxSplits = 8;        // of a chunk
constexpr int kMaxStepSplits = 32;   // of a decode step
constexpr int kMergeThreads = 256;

template <int D, int kW>
__global__ void __launch_bounds__(kMergeThreads)
prefill_mod_merge_kernel(const float *__restrict__ ws_o, const float *__restrict__ ws_lse,
                         int num_splits, const int32_t *__restrict__ cu_q, int T, int total_q,
                         int Hq, int G, int row_cap, __nv_bfloat16 *__restrict__ out) {
  constexpr int kRows = kMergeThreads / 32 / kW;  // rows of a block
  constexpr int kE = D / 32;                      // elements of a lane: 4 or 8
  __shared__ float s_acc[kW > 1 ? kMergeThreads / 32 : 1][D], s_w[kMergeThreads / 32];
  const int b = blockIdx.y;
  const int q0 = T > 0 ? b * T : cu_q[b], n_b = T > 0 ? T : cu_q[b + 1] - q0;
  if (n_b <= 0 || q0 < 0 || q0 + n_b > total_q) {  // no output rows (as in the attention)
    grid_dependency_wait();  // (a grid of such blocks alone must not end before the attention)
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % kW;
  const int64_t idx = (int64_t)blockIdx.x * kRows + warp / kW;  // token idx / Hq, head idx % Hq
  // only the rows the attention grid covers (tile rows i*G + g < row_cap)
  const bool live = idx < (int64_t)n_b * Hq && (idx / Hq) * G + (idx % Hq) % G < row_cap;
  const size_t row = (size_t)q0 * Hq + (live ? idx : 0);
  const size_t plane = (size_t)total_q * Hq;
  grid_dependency_wait();
  ws_o = after_wait(ws_o);
  ws_lse = after_wait(ws_lse);
  launch_dependents();  // (not before: the attention's SMs are free now)
  const float my_lse = live && lane < num_splits ? ws_lse[lane * plane + row] : -INFINITY;
  const float mx = warp_max(my_lse);  // (of the numbers among them)
  const float my_w = my_lse == -INFINITY ? 0.f : exp2f(my_lse - mx);
  float acc[kE], wsum = 0.f;
#pragma unroll
  for (int e = 0; e < kE; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int s = sub; s < num_splits; s += kW) {  // warp-uniform
    const float w = __shfl_sync(0xffffffffu, my_w, s);
    if (w == 0.f) continue;
    const float4 *src = reinterpret_cast<const float4 *>(ws_o + (s * plane + row) * D + kE * lane);
#pragma unroll
    for (int i = 0; i < kE / 4; ++i) {
      const float4 v = src[i];
      acc[4 * i] = fmaf(w, v.x, acc[4 * i]), acc[4 * i + 1] = fmaf(w, v.y, acc[4 * i + 1]);
      acc[4 * i + 2] = fmaf(w, v.z, acc[4 * i + 2]), acc[4 * i + 3] = fmaf(w, v.w, acc[4 * i + 3]);
    }
    wsum += w;
  }
  if constexpr (kW > 1) {
#pragma unroll
    for (int e = 0; e < kE; ++e) s_acc[warp][kE * lane + e] = acc[e];
    if (lane == 0) s_w[warp] = wsum;
    __syncthreads();
    if (sub != 0) return;
    for (int w = 1; w < kW; ++w) {
      wsum += s_w[warp + w];
#pragma unroll
      for (int e = 0; e < kE; ++e) acc[e] += s_acc[warp + w][kE * lane + e];
    }
  }
  if (!live) return;
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
  uint32_t ow[kE / 2];
#pragma unroll
  for (int e = 0; e < kE / 2; ++e) {
    __nv_bfloat162 b2 = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    ow[e] = *reinterpret_cast<uint32_t *>(&b2);
  }
  __nv_bfloat16 *dst = out + row * D + kE * lane;
  if constexpr (kE == 8)
    *reinterpret_cast<uint4 *>(dst) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
  else
    *reinterpret_cast<uint2 *>(dst) = make_uint2(ow[0], ow[1]);
}

template <int D, int kCopies, class Mod>
cudaError_t launch_d(const nvkv_cache &c, const nvkv_seqs &s, const void *q, const int32_t *cu_q,
                     int T, int total_q, int max_q, int Hq, float sm_scale, void *out,
                     int num_splits, float *ws_o, float *ws_lse, cudaStream_t stream,
                     const Mod &mod) {
  CUtensorMap map;
  if (!make_pool_tmap(c, &map)) return cudaErrorNotSupported;
  const int G = Hq / c.num_kv_heads;
  constexpr int kTileRows = 128 / kCopies;
  const int mtiles = (int)(((int64_t)max_q * G + kTileRows - 1) / kTileRows);
  constexpr int smem = Cfg<D>::kSmemBytes;
  cudaError_t e = cudaFuncSetAttribute(prefill_mod_kernel<D, kCopies, Mod>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  Args a;
  a.num_pages = c.num_pages, a.Hkv = c.num_kv_heads;
  a.page_table = s.page_table, a.max_pages = s.max_pages_per_seq;
  a.kv_lens = s.kv_lens, a.max_kv_len = s.max_kv_len;
  a.q = static_cast<const __nv_bfloat16 *>(q), a.cu_q = cu_q;
  a.T = T, a.total_q = total_q, a.Hq = Hq, a.qscale = sm_scale * kLog2e;
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.num_splits = num_splits;
  a.ws_o = num_splits > 1 ? ws_o : nullptr, a.ws_lse = ws_lse;
  a.err = s.err_word;
  const dim3 grid((unsigned)(mtiles * num_splits), (unsigned)c.num_kv_heads, (unsigned)s.batch);
  const DependentLaunch launch(grid, kThreads, smem, stream, true);
  e = cudaLaunchKernelEx(&launch.cfg, prefill_mod_kernel<D, kCopies, Mod>, map, (const Args)a, mod);
  if (e != cudaSuccess || num_splits == 1) return e;
  const int per_block = num_splits > 8 ? 1 : kMergeThreads / 32;
  const DependentLaunch merge(
      dim3((unsigned)(((int64_t)max_q * Hq + per_block - 1) / per_block), (unsigned)s.batch),
      kMergeThreads, 0, stream, true);
  return cudaLaunchKernelEx(
      &merge.cfg, num_splits > 8 ? prefill_mod_merge_kernel<D, 8> : prefill_mod_merge_kernel<D, 1>,
      (const float *)ws_o, (const float *)ws_lse, num_splits, cu_q, T, total_q, Hq, G,
      kTileRows * mtiles, static_cast<__nv_bfloat16 *>(out));
}

// Copies of the query rows in a tile: as many as fit when a sequence has one
// tile at most.
int copies_of(int max_q, int G) {
  const int64_t rows = (int64_t)max_q * G;
  return rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
}

template <class Mod>
cudaError_t launch_rows(const nvkv_cache &c, const nvkv_seqs &s, const void *q,
                        const int32_t *cu_q, int T, int total_q, int max_q, int Hq, float sm_scale,
                        void *out, int num_splits, float *ws_o, float *ws_lse, cudaStream_t stream,
                        const Mod &mod) {
  auto go = [&](auto copies) {
    constexpr int kCopies = decltype(copies)::value;
    return c.head_dim == 256
               ? launch_d<256, kCopies>(c, s, q, cu_q, T, total_q, max_q, Hq, sm_scale, out,
                                        num_splits, ws_o, ws_lse, stream, mod)
               : launch_d<128, kCopies>(c, s, q, cu_q, T, total_q, max_q, Hq, sm_scale, out,
                                        num_splits, ws_o, ws_lse, stream, mod);
  };
  const int copies = copies_of(max_q, Hq / c.num_kv_heads);
  if (copies == 4) return go(std::integral_constant<int, 4>{});
  if (copies == 2) return go(std::integral_constant<int, 2>{});
  return go(std::integral_constant<int, 1>{});
}

}  // namespace

// Key splits of a call with n query tiles (of all kv-heads and sequences): the
// count in 1 .. most with the least estimated time. A CTA takes about kSetup
// tiles' time before its first and after its last tile; n CTAs a split run in
// ceil(n S / SMs) waves; the merge of S fp32 planes of `values` outputs takes
// kMergeBytes a tile's time. Keys from documents (key_starts) are not known
// here: the splits of a chunk then only fill the first wave. The constants put
// the estimate within 1 % of the best count of each case that was swept (us):
//   65,536 + 2,048 tokens, 24/4 x 256, cap  1: 4233  3: 3842  4: 3975  5: 3825 (3)
//   65,536 + 100, the same heads            1: 1363  4: 356   7: 215   8: 352 (7)
//   20,000 + 300 and 9,000 + 150, the same  1: 539   4: 308   6: 303   8: 315 (6)
//   30,000 + 2,048, 16/4 x 128              1: 950   3: 973   4: 883   5: 917 (4)
//   731 of a prefix, 8/2 x 128              1: 26.7  2: 22.7  3: 22.5  4: 28.7 (3)
// (the count taken in brackets; chunks of few tiles, 2.2 to 2.6 waves, take 1).
static int estimate_splits(int64_t n, int64_t keys, int64_t values, bool first_wave, int most,
                           int sms) {
  constexpr double kSetup = 6.0, kMergeBytes = 6.0e6;
  const int64_t tiles = (keys + kTileTokens - 1) / kTileTokens;
  int best = 1;
  double least = 0;
  for (int S = 1; S <= most; ++S) {
    if (S > 1 && first_wave && n * S > sms) break;
    const double waves = (double)((n * S + sms - 1) / sms);
    double cost = waves * (kSetup + (double)((tiles + S - 1) / S));
    if (S > 1) cost += 2.0 + (double)values * (8.0 * S + 2.0) / kMergeBytes;
    if (S == 1 || cost < least) best = S, least = cost;
  }
  return best;
}

// Keys that a tile of `span` consecutive queries can see.
static int64_t visible_keys(const nvkv_seqs &s, const ScoreMod &mod, int span) {
  const int64_t w = (int64_t)mod.window + span + kTileTokens;  // (a prefix may add to it)
  return mod.window > 0 && w < s.max_kv_len ? w : s.max_kv_len;
}

int prefill_mod_auto_splits(const nvkv_cache &c, const nvkv_seqs &s, int total_q, int max_q,
                            int Hq, const ScoreMod &mod, int sms) {
  const int G = Hq / c.num_kv_heads;
  const int64_t n = ((int64_t)max_q * G + 127) / 128 * c.num_kv_heads * s.batch;
  return estimate_splits(n, visible_keys(s, mod, 128 / G), (int64_t)total_q * Hq * c.head_dim,
                         mod.starts != nullptr, kMaxSplits, sms);
}

cudaError_t launch_prefill_mod(const nvkv_cache &c, const nvkv_seqs &s, const void *q,
                               const int32_t *cu_q, int total_q, int max_q, int Hq,
                               float sm_scale, void *out, int num_splits, float *ws_o,
                               float *ws_lse, cudaStream_t stream, const ScoreMod &mod) {
  if (num_splits < 1 || num_splits > kMaxSplits || (num_splits > 1 && (!ws_o || !ws_lse)))
    return cudaErrorInvalidValue;
  return with_mod(mod, [&](const auto &m) {
    return launch_rows(c, s, q, cu_q, 0, total_q, max_q, Hq, sm_scale, out, num_splits, ws_o,
                       ws_lse, stream, m);
  });
}

// A decode step of T queries per sequence (T * Hq/Hkv <= 128 rows, one query
// tile for each kv-head and sequence). ws_o and ws_lse have room for `slots`
// partial results of a (sequence, kv-head) pair's rows each.
cudaError_t launch_decode_rows(const nvkv_cache &c, const nvkv_seqs &s, const void *q, int T,
                               int Hq, float sm_scale, int64_t slots, float *ws_o, float *ws_lse,
                               void *out, int sms, cudaStream_t stream, const ScoreMod &mod) {
  const int64_t n = (int64_t)c.num_kv_heads * s.batch;
  const int total_q = s.batch * T;
  const int room = (int)(slots / n < kMaxStepSplits ? slots / n : kMaxStepSplits);
  const int S = estimate_splits(n, visible_keys(s, mod, T), (int64_t)total_q * Hq * c.head_dim,
                                false, room > 1 ? room : 1, sms);
  return with_mod(mod, [&](const auto &m) {
    return launch_rows(c, s, q, nullptr, T, total_q, T, Hq, sm_scale, out, S, ws_o, ws_lse, stream,
                       m);
  });
}

}  // namespace nvkv
