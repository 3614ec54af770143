// The weight pass of kv_nvfp4_decode_attn_weights: what every query row of the call gave to each
// key, summed per key. The attention kernel before it (decode.cu or tile.cu) leaves each row's
// softmax statistics (m, 1 / l); with them a key's weight needs no further reduction over keys:
//   w_out[s][h][t] = w_in[s][h][t] + sum over the rows r of (s, h) that see t of
//                    exp2((q_r . k_t - m_r) c2) / l_r,     c2 = sm_scale log2(e).
//
// The scores are computed again from the K half of the cache (72 of a token's 144 bytes per KV
// head). The product is taken transposed, keys as the M dimension: a thread owns one key (its
// tensor-memory lane) and sums over the query rows in its own registers, in row order, so there is
// no reduction across threads and no atomic, and the result does not depend on the launch shape.
//
// A CTA takes `blocks_per_cta` consecutive 128-key blocks (two pages) of one (sequence, KV head), two
// at a time, and walks all row tiles of 48 rows over the pair: Q.K^T by tcgen05.mma
// kind::mxf4nvf4, M = 128 keys, N = the tile's rows (a multiple of 16 up to 48), two K = 64
// instructions per tile and block. A thread sums two keys, one of each block, so that the tile's
// statistics are read once for both and two independent chains run. Roles (256 threads): warp 0
// copies K pages (ring of kStages blocks), warp 1 issues the MMAs and owns tensor memory, warps 2, 3
// lay out Q tiles (codes in the tensor core's tile order, scales, statistics; ring of two, or a
// single tile loaded once when all rows fit one), warps 4..7 sum. Two such CTAs share an SM. Every
// wait is bounded in time, as in the attention kernels.
//
// Bounds. 48 rows over 4 x 100000 tokens, 4 KV heads: 115 MB of K and 13 MB of accounts, 19 us of HBM
// time; the call takes 107 us with the pass and 74 without it, most of the difference with the sums left
// out too (28). 384 rows over 2 x 32768 tokens: 0.1 G exponentials; 86 us with the pass, 50 without. Neither
// memory (43 % and 6 % of DRAM throughput) nor issue slots (45 % and 40 %) are full. Of the second
// call's 2.0K cycles per step and CTA, 0.8K are left when the warps only hand over (no product, load or
// sum), the MMAs add 0.5K, the loads nothing, the exponentials 0.3K, the statistics' loads and the rest
// of the sums 0.4K: hence two key blocks per step, one commit, and statistics read once for two keys.
// Tried and slower (us, the two calls; 110 / 99 then): tiles of 96 rows with two sets of summing warps
// 117 / 101, a second group of summing warps 112 / 99, a second MMA warp (and 8 columns at a time, for
// registers) 114 / 103, unpaired fp32 arithmetic 120 / 109, the S buffer released before its last sums
// 2 % more. The same: four slots for Q tiles, an issuing thread chosen by elect.sync, no suspending.

#include <cstdint>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"

namespace kvnvfp4 {

namespace {

constexpr int kStages = 8;
constexpr int kPair = 2;                     // key blocks of a step
constexpr int kRowTile = 48;                 // query rows of a tile
constexpr int kStScales = 8192;              // within a stage: K codes of two pages, then scales
constexpr int kStageBytes = 8192 + 2 * 1024;
constexpr int kQTileBytes = kRowTile * 64;
// a Q slot: codes, scale factors [2 k-halves][32 x 16 B], -m c2 [48], 1 / l [48]
constexpr int kQSf = kQTileBytes, kQNegM = kQSf + 1024, kQInv = kQNegM + kRowTile * 4;
constexpr int kQSlotBytes = kQInv + kRowTile * 4;

constexpr int kOffStage = 0;
constexpr int kOffSfk = kOffStage + kStages * kStageBytes;  // [kStages][2 k-halves][32 x 16 B]
constexpr int kOffQ = kOffSfk + kStages * 1024;             // [2] Q slots
constexpr int kOffBars = kOffQ + 2 * kQSlotBytes;
constexpr int kBarKFull = 0, kBarKEmpty = kBarKFull + kStages, kBarQFull = kBarKEmpty + kStages;
constexpr int kBarQEmpty = kBarQFull + 2, kBarSFull = kBarQEmpty + 2, kBarSEmpty = kBarSFull + 2;
constexpr int kBarDrain = kBarSEmpty + 2, kNumBars = kBarDrain + 1;
constexpr int kOffTmemSlot = kOffBars + kNumBars * 8;
constexpr int kSmemBytes = kOffTmemSlot + 16;
static_assert(kQTileBytes % 16 == 0 && kQSlotBytes % 16 == 0 && kOffBars % 8 == 0, "alignment");

// tensor memory: S [2][kPair][48], K scales [2][kPair][2 k-halves][4], Q scales [2][2 k-halves][4]
constexpr uint32_t kColS = 0, kColSfa = 192, kColSfb = 224, kTmemCols = 256;
constexpr int kCtasPerSm = 2;
static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of two CTAs");

constexpr int kWarpProducer = 0, kWarpMma = 1, kWarpQ0 = 2, kWarpSum0 = 4;
constexpr int kSumWarps = 4;
constexpr int kThreads = 32 * (kWarpSum0 + kSumWarps);

struct WeightParams {
  const uint8_t* q_codes;
  const uint8_t* q_scales;
  const uint8_t* pool;
  const int32_t* block_table;
  const int4* groups;      // 2 x int4 per group, .w of the first = the sequence's length
  const float2* stats;     // [num_seqs][Hkv][rows]: m, 1 / l
  const float* w_in;       // [num_seqs][Hkv][w_stride], or null for zeros
  float* w_out;
  int64_t w_stride;
  int32_t max_pages, num_pages;
  int32_t groups_per_seq;
  int32_t Hq, Hkv, G, q_len, rows, causal;
  int32_t chunks, blocks_per_cta;  // CTAs per (sequence, KV head), blocks of each
  int32_t* status;
  float c2;
};

// What one CTA works on.
struct Span {
  int seq, head, len, b0, b1, tiles;
  __device__ Span(const WeightParams& p) {
    head = blockIdx.x % p.Hkv;
    const int rest = blockIdx.x / p.Hkv;
    seq = rest / p.chunks;
    len = p.groups[2 * ((int64_t)seq * p.groups_per_seq)].w;
    b0 = (rest % p.chunks) * p.blocks_per_cta;
    b1 = min(b0 + p.blocks_per_cta, (len + 127) >> 7);
    tiles = (p.rows + kRowTile - 1) / kRowTile;
  }
  // the first row tile with a row that sees the block's first key
  __device__ int first_tile(const WeightParams& p, int b) const {
    const int64_t t = (int64_t)b * 128 - (len - p.q_len);
    return p.causal && t > 0 ? (int)(t * p.G / kRowTile) : 0;
  }
};

__device__ __forceinline__ void produce_keys(const WeightParams& p, const Span& sp, uint32_t sbase,
                                             int lane) {
  const uint32_t bars = sbase + kOffBars;
  const bool lone = (sp.head | 1) >= p.Hkv;  // the last head of an odd count has no partner
  const uint32_t ksb = lone ? 512u : 1024u;
  const int32_t* bt = p.block_table + (int64_t)sp.seq * p.max_pages;
  const int pages = (sp.len + kPage - 1) / kPage;
  uint32_t k = 0;
  bool to = false;
  for (int b = sp.b0; b < sp.b1; b += 16) {
    const int page = 2 * b + lane;
    const int32_t mine = page < pages ? bt[page] : -1;
    for (int j = 0; j < 16 && b + j < sp.b1; ++j, ++k) {
      const int32_t pid[2] = {__shfl_sync(0xffffffffu, mine, 2 * j),
                              __shfl_sync(0xffffffffu, mine, 2 * j + 1)};
      if (lane == 0) {
        const uint32_t st = k % kStages, full = bars + 8 * (kBarKFull + st);
        if (k >= kStages)
          wait_bar_sleep(bars + 8 * (kBarKEmpty + st), ((k / kStages) - 1) & 1, to);
        uint32_t bytes = 0;
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (pid[q] >= 0 && pid[q] < p.num_pages) bytes += 4096u + ksb;
        if (bytes == 0) {
          mbar_arrive(full);
        } else {
          mbar_arrive_expect_tx(full, bytes);
          const uint32_t dst = sbase + kOffStage + st * kStageBytes;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (pid[q] < 0 || pid[q] >= p.num_pages) continue;
            const uint8_t* src = p.pool + (int64_t)pid[q] * p.Hkv * 9216;
            bulk_g2s(dst + q * 4096, src + sp.head * 4096, 4096u, full);
            bulk_g2s(dst + kStScales + q * 1024, src + p.Hkv * 4096 + (sp.head >> 1) * 1024, ksb,
                     full);
          }
        }
      }
      __syncwarp();
    }
  }
  if (lane == 0) {
    // no copy into this CTA's shared memory may still be in flight at exit
    for (uint32_t st = 0; st < kStages && st < k; ++st) {
      const uint32_t last = k - 1 - ((k - 1 - st) % kStages);
      wait_bar_sleep(bars + 8 * (kBarKFull + st), (last / kStages) & 1, to);
    }
    if (to) flag_status(p.status, KV_NVFP4_DEV_TIMEOUT);
  }
}

// The rows lane and lane + 32 of a row tile (48 rows: the upper half of the lanes has one).
struct QRows {
  uint4 c[2][4];
  uint2 sc[2];
  float2 st[2];
};

__device__ __forceinline__ void fetch_q_tile(const WeightParams& p, const Span& sp, int tile,
                                             int lane, QRows& q) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = lane + 32 * u, r = tile * kRowTile + i;
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) q.c[u][ch] = make_uint4(0u, 0u, 0u, 0u);
    q.sc[u] = make_uint2(0u, 0u);
    q.st[u] = make_float2(0.f, 0.f);
    if (i >= kRowTile || r >= p.rows) continue;
    const int64_t qrow = ((int64_t)sp.seq * p.q_len + r / p.G) * p.Hq + sp.head * p.G + r % p.G;
    const uint4* src = reinterpret_cast<const uint4*>(p.q_codes + qrow * kCodeBytes);
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) q.c[u][ch] = src[ch];
    q.sc[u] = *reinterpret_cast<const uint2*>(p.q_scales + qrow * kScaleBytes);
    q.st[u] = p.stats[((int64_t)sp.seq * p.Hkv + sp.head) * p.rows + r];
  }
}

__device__ __forceinline__ void store_q_tile(const WeightParams& p, uint8_t* slot, int lane,
                                             const QRows& q) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = lane + 32 * u;
    if (i >= kRowTile) continue;
#pragma unroll
    for (int ch = 0; ch < 4; ++ch)
      *reinterpret_cast<uint4*>(slot + (i >> 3) * 512 + ch * 128 + (i & 7) * 16) = q.c[u][ch];
    // a row past the last, or one that saw no key at all, adds nothing: exp2(-inf) * 0
    const bool live = q.st[u].y > 0.f;
    reinterpret_cast<float*>(slot + kQNegM)[i] = live ? -(q.st[u].x * p.c2) : -INFINITY;
    reinterpret_cast<float*>(slot + kQInv)[i] = live ? q.st[u].y : 0.f;
  }
  // scale-factor rows: row `lane` holds the 4-byte groups of tile rows lane and 32 + lane (and zeros
  // for the rows from 48 on that a wider tile would have)
#pragma unroll
  for (int kh = 0; kh < 2; ++kh)
    *reinterpret_cast<uint4*>(slot + kQSf + kh * 512 + lane * 16) =
        make_uint4(kh ? q.sc[0].y : q.sc[0].x, kh ? q.sc[1].y : q.sc[1].x, 0u, 0u);
}

// The two Q warps take alternate steps, each with a slot of its own, and fetch their next tile
// before they wait for the slot: a fetch takes about as long as the sums of two steps.
__device__ __forceinline__ void load_queries(const WeightParams& p, const Span& sp, uint8_t* smem,
                                             int warp, int lane) {
  const uint32_t bars = smem_u32(smem) + kOffBars;
  const uint32_t sl = (uint32_t)(warp - kWarpQ0);
  uint8_t* slot = smem + kOffQ + sl * kQSlotBytes;
  int b = sp.b0, tile = b < sp.b1 ? sp.first_tile(p, b) : 0;
  auto next = [&]() {
    if (++tile == sp.tiles && (b += kPair) < sp.b1) tile = sp.first_tile(p, b);
  };
  if (sp.tiles == 1 && sl == 1) return;  // the one tile stays in slot 0
  if (sl == 1 && b < sp.b1) next();
  QRows q;
  if (b < sp.b1) fetch_q_tile(p, sp, tile, lane, q);
  uint32_t use = 0;
  bool to = false;
  while (b < sp.b1) {
    if (use > 0) wait_bar_sleep(bars + 8 * (kBarQEmpty + sl), (use - 1) & 1, to);
    store_q_tile(p, slot, lane, q);
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * (kBarQFull + sl));
    if (sp.tiles == 1) return;
    ++use;
    next();
    if (b < sp.b1) next();
    if (b < sp.b1) fetch_q_tile(p, sp, tile, lane, q);
  }
  if (to && lane == 0) flag_status(p.status, KV_NVFP4_DEV_TIMEOUT);
}

__device__ __forceinline__ uint64_t desc_add(uint64_t d, uint32_t bytes) {
  return d + (uint64_t)(bytes >> 4);  // start-address field: addresses stay below 2^18
}

__device__ __forceinline__ void issue_products(const WeightParams& p, const Span& sp,
                                               uint32_t sbase, uint32_t tbase, int lane) {
  const uint32_t bars = sbase + kOffBars;
  const bool lone = (sp.head | 1) >= p.Hkv;
  const bool one = sp.tiles == 1;
  const uint32_t n = one ? (uint32_t)((p.rows + 15) & ~15) : (uint32_t)kRowTile;
  // A, B = E2M1 K-major, scale type UE4M3, M = 128
  const uint32_t idesc = (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((128u >> 4) << 24);
  const uint64_t dk = smem_desc(sbase + kOffStage, 128, 512);
  const uint64_t dq = smem_desc(sbase + kOffQ, 128, 512);
  const uint64_t dsfk = smem_desc(sbase + kOffSfk, 16, 128);
  const uint64_t dsfq = smem_desc(sbase + kOffQ + kQSf, 16, 128);
  uint32_t k = 0, step = 0;
  bool to = false;
  for (int b = sp.b0; b < sp.b1; b += kPair, k += kPair) {
    const int blocks = min(kPair, sp.b1 - b);
    for (int i = 0; i < blocks; ++i) {
      const uint32_t st = (k + i) % kStages;
      const uint32_t stage = sbase + kOffStage + st * kStageBytes;
      wait_bar_sleep(bars + 8 * (kBarKFull + st), ((k + i) / kStages) & 1, to);
      // the head's K scales of both pages into the scale-factor copy's rows: row r = page 0's keys r
      // and r + 32, then page 1's. The slot's previous reader completed before the stage was refilled
#pragma unroll
      for (int kh = 0; kh < 2; ++kh) {
        uint2 v[2];
#pragma unroll
        for (int q = 0; q < 2; ++q)  // a skipped page leaves stale scales: its keys are not counted
          v[q] = lone
                     ? lds64(stage + kStScales + q * 1024 + kh * 256 + lane * 8)
                     : lds64(stage + kStScales + q * 1024 + kh * 512 + lane * 16 + (sp.head & 1) * 8);
        sts128(sbase + kOffSfk + st * 1024 + kh * 512 + lane * 16, v[0].x, v[0].y, v[1].x, v[1].y);
      }
    }
    fence_async_smem();
    __syncwarp();
    bool fresh = true;  // the pair's scales are not in tensor memory yet
    for (int tile = sp.first_tile(p, b); tile < sp.tiles; ++tile, ++step) {
      const uint32_t buf = step & 1u, sl = one ? 0u : buf;
      // S buffer `buf` and the Q scales beside it are free once step - 2 has been read; so are the
      // K scales of the pair before the last, whose last step was step - 2 or earlier
      if (step >= 2) wait_bar_sleep(bars + 8 * (kBarSEmpty + buf), ((step >> 1) - 1) & 1, to);
      if (!one || step == 0)
        wait_bar_sleep(bars + 8 * (kBarQFull + sl), one ? 0u : (step >> 1) & 1, to);
      if (to) break;
      if (lane == 0) {
        tc_fence_after();
        const uint32_t sfb = tbase + kColSfb + sl * 8;
        const uint64_t qd = desc_add(dq, sl * kQSlotBytes);
        if (!one || step == 0) {
          tmem_cp_32x128b_x4(sfb, desc_add(dsfq, sl * kQSlotBytes));
          tmem_cp_32x128b_x4(sfb + 4, desc_add(dsfq, sl * kQSlotBytes + 512));
        }
        for (int i = 0; i < blocks; ++i) {
          const uint32_t st = (k + i) % kStages;
          const uint32_t sfa = tbase + kColSfa + ((k & 2u) + i) * 8;
          const uint32_t d = tbase + kColS + (2 * buf + i) * kRowTile;
          const uint64_t kd = desc_add(dk, st * kStageBytes);
          if (fresh) {
            tmem_cp_32x128b_x4(sfa, desc_add(dsfk, st * 1024));
            tmem_cp_32x128b_x4(sfa + 4, desc_add(dsfk, st * 1024 + 512));
          }
          mma_nvf4_ss(d, kd, qd, idesc, sfa, sfb, 0u);
          mma_nvf4_ss(d, desc_add(kd, 256), desc_add(qd, 256), idesc, sfa + 4, sfb + 4, 1u);
        }
        // the only commit: the summing warps, which wait for it, release the Q slot and the K stages
        // (a tcgen05 instruction costs this warp 100 to 200 cycles, and it is the one that never waits)
        mma_commit(bars + 8 * (kBarSFull + buf));
      }
      fresh = false;
      __syncwarp();
    }
    if (to) break;
  }
  if (to && lane == 0) flag_status(p.status, KV_NVFP4_DEV_TIMEOUT);
}

// Adds 16 rows' exp2(s c2 - m c2) / l for each of the thread's two keys. The product m c2 is rounded
// once per row, as in the tile kernel's P, whose sum l divides by: the two roundings cancel.
// kMasked: only rows from r0 on see a key.
template <bool kMasked>
__device__ __forceinline__ void add_rows16(const uint32_t (&s)[kPair][16], const float* negm,
                                           const float* inv, uint64_t c2, const int (&r0)[kPair],
                                           int c0, uint64_t (&acc)[kPair][2]) {
#pragma unroll
  for (int c = 0; c < 16; c += 4) {
    const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(negm + c);
    const ulonglong2 iv = *reinterpret_cast<const ulonglong2*>(inv + c);
#pragma unroll
    for (int i = 0; i < kPair; ++i)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        float x, y;
        halves_of(fma2(pair_of(__uint_as_float(s[i][c + e]), __uint_as_float(s[i][c + e + 1])), c2,
                       e ? m.y : m.x),
                  x, y);
        x = fast_exp2(x);
        y = fast_exp2(y);
        if (kMasked) {
          x = c0 + c + e >= r0[i] ? x : 0.f;
          y = c0 + c + e + 1 >= r0[i] ? y : 0.f;
        }
        acc[i][e / 2] = fma2(pair_of(x, y), e ? iv.y : iv.x, acc[i][e / 2]);
      }
  }
}

__device__ __forceinline__ void sum_weights(const WeightParams& p, const Span& sp, uint8_t* smem,
                                            uint32_t tbase, int warp, int lane) {
  const uint32_t bars = smem_u32(smem) + kOffBars;
  const int q = warp & 3, key = 32 * q + lane;
  const bool one = sp.tiles == 1;
  const int cols = one ? (p.rows + 15) & ~15 : kRowTile;
  const int32_t* bt = p.block_table + (int64_t)sp.seq * p.max_pages;
  const int64_t wrow = ((int64_t)sp.seq * p.Hkv + sp.head) * p.w_stride;
  const uint32_t scol = tbase + ((uint32_t)(32 * q) << 16) + kColS;
  const uint64_t c2 = pair_of(p.c2, p.c2);
  const int L0 = sp.len - p.q_len;
  uint32_t step = 0;
  bool to = false;
  for (int b = sp.b0; b < sp.b1; b += kPair) {
    int first[kPair];
    bool real[kPair], valid[kPair];
    float before[kPair];
#pragma unroll
    for (int i = 0; i < kPair; ++i) {
      const int t = (b + i) * 128 + key;
      real[i] = b + i < sp.b1 && t < sp.len;
      // (a plain load: a kernel that this one was launched beside may have written the table)
      const int32_t pid = real[i] ? bt[t / kPage] : -1;
      valid[i] = pid >= 0 && pid < p.num_pages;  // a bad page's keys got no weight
      before[i] = real[i] && p.w_in != nullptr ? p.w_in[wrow + t] : 0.f;
      first[i] = p.causal && t > L0 ? (t - L0) * p.G : 0;  // the first row that sees the key
    }
    // the first row that sees the pair's last key: a tile from there on is seen whole
    const int last = (b + kPair) * 128 - 1;
    const int whole = p.causal && last > L0 ? (last - L0) * p.G : 0;
    uint64_t acc[kPair][2] = {};
    for (int tile = sp.first_tile(p, b); tile < sp.tiles; ++tile, ++step) {
      const uint32_t buf = step & 1u;
      const uint8_t* slot = smem + kOffQ + (one ? 0u : buf) * kQSlotBytes;
      const float* negm = reinterpret_cast<const float*>(slot + kQNegM);
      const float* inv = reinterpret_cast<const float*>(slot + kQInv);
      // the tile's statistics were written before its MMAs were issued, by other threads
      if (!one || step == 0)
        wait_bar_sleep(bars + 8 * (kBarQFull + (one ? 0u : buf)), one ? 0u : (step >> 1) & 1, to);
      wait_bar_sleep(bars + 8 * (kBarSFull + buf), (step >> 1) & 1, to);
      tc_fence_after();
      __syncwarp();
      const bool masked = whole > tile * kRowTile;
      int r0[kPair];
#pragma unroll
      for (int i = 0; i < kPair; ++i) r0[i] = first[i] - tile * kRowTile;
      const uint32_t col = scol + buf * (kPair * kRowTile);
      auto load = [&](uint32_t (&s)[kPair][16], int c) {
        tmem_ld16(col + c, s[0]);
        tmem_ld16(col + kRowTile + c, s[1]);
      };
      auto add = [&](uint32_t (&s)[kPair][16], int c) {
        if (masked) add_rows16<true>(s, negm + c, inv + c, c2, r0, c, acc);
        else add_rows16<false>(s, negm + c, inv + c, c2, r0, c, acc);
      };
      auto wait = [&](uint32_t (&s)[kPair][16]) {
        tmem_wait_ld_regs16(s[0]);
        tmem_wait_ld_regs16(s[1]);
      };
      // the tile's columns 16 at a time, the next 16 on their way while these are summed
      uint32_t s0[kPair][16], s1[kPair][16];
      load(s0, 0);
      wait(s0);
      if (cols > 16) load(s1, 16);
      add(s0, 0);
      if (cols > 16) {
        wait(s1);
        if (cols > 32) load(s0, 32);
        add(s1, 16);
        if (cols > 32) {
          wait(s0);
          add(s0, 32);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bars + 8 * (kBarSEmpty + buf));
        if (!one) mbar_arrive(bars + 8 * (kBarQEmpty + buf));
        if (tile + 1 == sp.tiles)  // the pair's products are complete, its K consumed
          for (int i = 0; i < min(kPair, sp.b1 - b); ++i)
            mbar_arrive(bars + 8 * (kBarKEmpty + (uint32_t)(b - sp.b0 + i) % kStages));
      }
    }
#pragma unroll
    for (int i = 0; i < kPair; ++i)
      if (real[i]) {
        float a[4];
        halves_of(acc[i][0], a[0], a[1]);
        halves_of(acc[i][1], a[2], a[3]);
        p.w_out[wrow + (b + i) * 128 + key] =
            valid[i] ? before[i] + ((a[0] + a[1]) + (a[2] + a[3])) : before[i];
      }
  }
  if (to && lane == 0) flag_status(p.status, KV_NVFP4_DEV_TIMEOUT);
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) weight_kernel(const WeightParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem), bars = sbase + kOffBars;
  asm volatile("griddepcontrol.launch_dependents;");
  // a sequence shorter than the longest has CTAs without blocks; the plan's tables were written
  // before the attention kernel started, so that they can be read ahead of the wait
  const Span sp(p);
  if (sp.b0 >= sp.b1) return;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bars + 8 * (kBarKFull + s), 1);
      mbar_init(bars + 8 * (kBarKEmpty + s), kSumWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bars + 8 * (kBarQFull + b), 1);
      mbar_init(bars + 8 * (kBarQEmpty + b), kSumWarps);
      mbar_init(bars + 8 * (kBarSFull + b), 1);
      mbar_init(bars + 8 * (kBarSEmpty + b), kSumWarps);
    }
    mbar_init(bars + 8 * kBarDrain, 1);
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(sbase + kOffTmemSlot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // a programmatic dependent of the attention kernel or its merge, which write the statistics
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(smem + kOffTmemSlot);
  if (warp == kWarpProducer) {
    produce_keys(p, sp, sbase, lane);
  } else if (warp == kWarpMma) {
    issue_products(p, sp, sbase, tbase, lane);
  } else if (warp < kWarpSum0) {
    load_queries(p, sp, smem, warp, lane);
  } else {
    sum_weights(p, sp, smem, tbase, warp, lane);
  }
  if (warp == kWarpMma) {
    // tensor memory is freed only once no tcgen05 op of this CTA is in flight
    if (lane == 0) mma_commit(bars + 8 * kBarDrain);
    __syncwarp();
    bool to = false;
    wait_bar_sleep(bars + 8 * kBarDrain, 0, to);
    if (to && lane == 0) flag_status(p.status, KV_NVFP4_DEV_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tbase, kTmemCols);
}

}  // namespace

cudaError_t launch_weights(const uint8_t* q_codes, const uint8_t* q_scales, const uint8_t* pool,
                           const int32_t* block_table, int32_t max_pages, int32_t num_pages,
                           const void* groups, int32_t groups_per_seq, int32_t num_seqs,
                           int32_t max_seq_len, int64_t total_tokens, const float2* stats,
                           const float* w_in, float* w_out, int64_t w_stride, int32_t Hq,
                           int32_t Hkv, int32_t q_len, int32_t causal, float sm_scale,
                           int32_t num_sms, int32_t* status, cudaStream_t stream) {
  static bool attr_done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  if (dev < 0 || dev >= 64 || !attr_done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        weight_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev] = true;
  }
  WeightParams p;
  p.q_codes = q_codes; p.q_scales = q_scales; p.pool = pool; p.block_table = block_table;
  p.groups = static_cast<const int4*>(groups); p.stats = stats;
  p.w_in = w_in; p.w_out = w_out; p.w_stride = w_stride;
  p.max_pages = max_pages; p.num_pages = num_pages; p.groups_per_seq = groups_per_seq;
  p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.q_len = q_len; p.rows = p.G * q_len;
  p.causal = causal; p.status = status;
  p.c2 = sm_scale * 1.4426950408889634f;
  // about one round of CTAs: each starts its pipeline once
  const int64_t blocks = (total_tokens / 128 + num_seqs) * Hkv;
  const int64_t places = (int64_t)num_sms * kCtasPerSm;
  const int64_t per = (blocks + places - 1) / places;
  p.blocks_per_cta = (int32_t)(per < 1 ? 1 : per > 256 ? 256 : per);
  const int64_t most = ((int64_t)max_seq_len + 127) / 128;
  p.chunks = (int32_t)((most + p.blocks_per_cta - 1) / p.blocks_per_cta);
  const int64_t grid = (int64_t)p.chunks * Hkv * num_seqs;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weight_kernel, p);
}

}  // namespace kvnvfp4
