// Eviction from the paged cache by accumulated attention weight: the choice of the slots to keep
// (kv_nvfp4_evict_select) and the compaction of the cache to them (kv_nvfp4_evict_compact).
//
// Select. Per set of slots (a KV head's, or a sequence's when all heads share one set) the slots
// [0, sink) and [len - recent, len) come first, by slot, then the rest by weight, ties to the lowest slot;
// the first min(len, keep) of that order are listed in ascending slot order. The weights are mapped
// to unsigned keys of the same order (NaN to 0, below every value) and the smallest kept key is
// found by a radix select.
//
// Compact. Row j of a set's new cache is row index[j] of its old one. The index ascends, so
// index[j] >= j and a tile of rows is written only over rows that no later tile reads: tiles in
// order, each read whole before it is written, compact the cache in place.

#include <cstdint>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"

namespace kvnvfp4 {

namespace {

struct SelectParams {
  const float* weights;    // [num_seqs][Hkv][w_stride]
  int64_t w_stride;
  const int32_t* seq_lens;
  const int32_t* keep;
  int32_t* index;          // [num_seqs][Hkv or 1][index_stride]
  int64_t index_stride;
  int32_t Hkv, per_head, sink, recent;
  int32_t cached;          // keys that fit a CTA's shared memory
  int32_t* status;
};

// Unsigned key in the order of the weights: NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t b = __float_as_uint(__fadd_rn(w, 0.0f));
  return w != w ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// The weight of a slot for a set: its head's, or the heads' sum (fp32, head after head).
__device__ __forceinline__ float set_weight(const float* w, int64_t stride, int heads, int64_t t) {
  float v = w[t];
  for (int h = 1; h < heads; ++h) v = __fadd_rn(v, w[(int64_t)h * stride + t]);
  return v;
}

// One cluster of C CTAs per set; a CTA takes a contiguous slice of the candidates [lo, hi) and keeps
// its keys in shared memory (what does not fit is read and mapped again from global memory in every
// pass). The radix select runs on the keys' distance from the smallest one, and its first digit is
// the top 11 bits of the largest distance: accumulated weights share a sign and most exponent bits,
// and with a digit of fixed bits a warp's 32 counts fell into a few bins and were serialised.
//
// Per pass each CTA counts its keys' digits in a shared histogram of 2048 bins and its sums over 64
// bins; the cluster meets; every CTA reads the C coarse histograms through distributed shared
// memory, finds the 64 bins that hold the need-th largest key, and reads those of every CTA (all C
// whole histograms are C x 8 KB for every CTA, which took 5 to 8 us). Once the chosen bin holds at
// most 2048 keys, which is after the first pass for weights that are not mostly equal, the CTAs
// exchange those keys instead, and each finds the threshold among them on its own, seven bits at a
// time until one key is left.
// With the exchanged keys go the counts of keys above the bin, so every CTA also knows how many
// slots the CTAs before it list: three meetings of the cluster in all. The warps then list their
// parts of the slice in order, by ballots.
//
// Bounds: the weights are read once (8.4 MB for 4 sequences x 4 KV heads x 131072 slots: 1.2 us of
// HBM time), but the passes over the cached keys, each a few instructions per key on the few SMs of
// a cluster, and the meetings follow one another: load 4 us, digit 1 and its sum 4, exchange and
// search 6, listing 2.5 of that case's 20.0 us (the launch and the clusters' start are the rest).
// One CTA per set without a cluster took 386 us there (2838 us for one set of 600000 slots and four
// heads, now 28 us).
constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048, kCoarse = kBins / 64;
constexpr int kSelMaxCluster = 16;
constexpr int kSelMaxCached = 48 * 1024;  // keys in shared memory (192 KB)
constexpr uint32_t kSelExchange = kBins;  // keys exchanged at most: they take the histograms' place
constexpr int kSelRounds = kSelExchange / kSelThreads;
static_assert(kSelThreads == kCoarse * kSelMaxCluster, "a thread per coarse bin and CTA");
static_assert(kCoarse == 32 && kSelWarps <= 32, "a lane per coarse bin, a lane per warp");

struct alignas(16) SelectShared {
  uint32_t hist[2][kBins];  // digit counts, alternating by pass: the peers may still read one
  uint32_t coarse[2][kCoarse];
  uint32_t all[kSelMaxCluster][64];  // counts read from the cluster
  uint32_t bins7[2][128];            // the search among the exchanged keys
  int32_t list_at[kSelExchange];     // where in the slice this CTA's exchanged keys are
  uint32_t lowest[kSelWarps], highest[kSelWarps];
  uint32_t digit, above, in_bin;
  int32_t warp_over[32], warp_tied[32];  // keys above the edge and equal to it, per warp's part
  // of the CTA, read by the cluster
  uint32_t low, high;
  uint32_t over;            // its keys above the digits found so far
  uint32_t listed;          // its keys that share them
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word at this CTA's shared address `a`, of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_peer(uint32_t a, uint32_t rank) {
  uint32_t remote;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(a), "r"(rank));
  return remote;
}
__device__ __forceinline__ uint32_t cluster_load(uint32_t remote) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

// Four weights from slot t on (16-byte aligned when kVec); slots from `end` on read as 0.
template <bool kVec>
__device__ __forceinline__ float4 load_weights4(const float* w, int64_t t, int64_t end) {
  if (kVec && t + 4 <= end) return *reinterpret_cast<const float4*>(w + t);
  return make_float4(t < end ? w[t] : 0.f, t + 1 < end ? w[t + 1] : 0.f,
                     t + 2 < end ? w[t + 2] : 0.f, t + 3 < end ? w[t + 3] : 0.f);
}

__device__ __forceinline__ float4 add4(const float4& a, const float4& b) {
  return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z),
                     __fadd_rn(a.w, b.w));
}

// kVec: the accounts' rows are 16-byte aligned
template <bool kVec>
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  SelectShared& sh = *reinterpret_cast<SelectShared*>(smem);
  uint32_t* cache = reinterpret_cast<uint32_t*>(smem + sizeof(SelectShared));
  const uint32_t C = cluster_size(), rank = cluster_rank();
  const int sets = p.per_head ? p.Hkv : 1;
  const int64_t unit = blockIdx.x / C;
  const int64_t seq = unit / sets;
  const int set = (int)(unit % sets);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 2 * kBins; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
  if (tid < 256) (&sh.bins7[0][0])[tid] = 0;
  if (tid == 0) sh.over = sh.listed = 0u;
  // Launched as a programmatic dependent of the kernel before it on the stream, which may have written
  // the weights or lengths: started while that one ends, 2 to 3 us per call. Neither kernel of this
  // file lets the next one start before its own end: clusters placed beside a running grid were packed
  // unevenly over the SMs (16 sets of 131072 slots 22.8 us, 20.0 so).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int32_t len = p.seq_lens[seq], keep = p.keep[seq];
  const int32_t kept = min(len, keep);
  // the exits below are the same for every CTA of the cluster
  if (len < 0 || keep < 0 || len > p.w_stride || kept > p.index_stride) {
    if (tid == 0 && rank == 0) flag_status(p.status, KV_NVFP4_DEV_BAD_POS);
    return;
  }
  int32_t* out = p.index + unit * p.index_stride;
  const float* w = p.weights + (seq * p.Hkv + set) * p.w_stride;
  const int heads = p.per_head ? 1 : p.Hkv;
  const int32_t step = (int32_t)C * kSelThreads, first = (int32_t)rank * kSelThreads + tid;
  // [lo, hi): the slots that are not protected
  const int32_t lo = min(len, p.sink), hi = max(lo, p.recent < len ? len - p.recent : 0);
  if (kept == len || lo + (len - hi) >= kept) {  // no choice by weight: the first kept of them
    for (int64_t j = first; j < kept; j += step)
      out[j] = kept == len || j < lo ? (int32_t)j : (int32_t)(hi + (j - lo));
    return;
  }
  const int32_t need = kept - lo - (len - hi);  // 1 <= need < hi - lo
  // this CTA's slice, slots t0 .. t0 + n - 1 less those below lo; slices start at multiples of 32
  const int32_t base = lo & ~31;
  const int32_t slice = (int32_t)((((int64_t)(hi - base) + C - 1) / C + 31) & ~31);
  const int32_t t0 = (int32_t)min((int64_t)hi, base + (int64_t)rank * slice);
  const int32_t n = min(slice, hi - t0), i_lo = max(0, lo - t0);
  const int32_t cached = min(n, p.cached);
  auto key_at = [&](int32_t i) {
    return i < cached ? cache[i] : order_key(set_weight(w, p.w_stride, heads, t0 + i));
  };

  // the slice's keys, the smallest and the largest
  uint32_t low = 0xFFFFFFFFu, high = 0u;
  auto take4 = [&](const float4& v, int32_t i) {
    const uint32_t k[4] = {order_key(v.x), order_key(v.y), order_key(v.z), order_key(v.w)};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i + e >= i_lo && i + e < n) {
        low = min(low, k[e]);
        high = max(high, k[e]);
      }
    }
    if (i + 4 <= cached) *reinterpret_cast<uint4*>(cache + i) = make_uint4(k[0], k[1], k[2], k[3]);
    else
      for (int e = 0; e < 4; ++e)
        if (i + e < cached) cache[i + e] = k[e];
  };
  // eight 16-byte loads in flight per thread: eight places, or two places of four heads; the last
  // places, and the heads behind a multiple of four, one by one
  int32_t i0 = 4 * tid;
  if (heads == 1) {
    for (; kVec && i0 + 28 * kSelThreads + 4 <= n; i0 += 32 * kSelThreads) {
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = *reinterpret_cast<const float4*>(w + t0 + i0 + u * 4 * kSelThreads);
#pragma unroll
      for (int u = 0; u < 8; ++u) take4(v[u], i0 + u * 4 * kSelThreads);
    }
  } else if (heads % 4 == 0) {
    for (; kVec && i0 + 4 * kSelThreads + 4 <= n; i0 += 8 * kSelThreads) {
      float4 sum[2];
      for (int h0 = 0; h0 < heads; h0 += 4) {
        float4 v[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int h = 0; h < 4; ++h)
            v[u][h] = *reinterpret_cast<const float4*>(w + (h0 + h) * p.w_stride + t0 + i0 +
                                                       u * 4 * kSelThreads);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int h = 0; h < 4; ++h) sum[u] = h0 + h == 0 ? v[u][h] : add4(sum[u], v[u][h]);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) take4(sum[u], i0 + u * 4 * kSelThreads);
    }
  }
  for (; i0 < n; i0 += 4 * kSelThreads) {
    float4 sum = load_weights4<kVec>(w, (int64_t)t0 + i0, hi);
    for (int h = 1; h < heads; ++h)
      sum = add4(sum, load_weights4<kVec>(w + h * p.w_stride, (int64_t)t0 + i0, hi));
    take4(sum, i0);
  }
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) {
    sh.lowest[warp] = low;
    sh.highest[warp] = high;
  }
  __syncthreads();
  if (warp == 0) {
    low = __reduce_min_sync(0xffffffffu, lane < kSelWarps ? sh.lowest[lane] : 0xFFFFFFFFu);
    high = __reduce_max_sync(0xffffffffu, lane < kSelWarps ? sh.highest[lane] : 0u);
    if (lane == 0) {
      sh.low = low;
      sh.high = high;
    }
  }
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  low = lane < C ? cluster_load(cluster_peer(smem_u32(&sh.low), lane)) : 0xFFFFFFFFu;
  high = lane < C ? cluster_load(cluster_peer(smem_u32(&sh.high), lane)) : 0u;
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);

  // The candidates from place `from` to `to`, in steps of `threads` threads of which this is thread
  // `me`: four at a time where they lie in the cache.
  auto each_key = [&](int32_t from, int32_t to, int me, int threads, auto&& f) {
    const int32_t b4 = min(to, cached) & ~3, a4 = min((from + 3) & ~3, max(b4, from));
    for (int32_t i = from + me; i < min(a4, to); i += threads) f(key_at(i), i);
#pragma unroll 2
    for (int32_t i = a4 + 4 * me; i < b4; i += 4 * threads) {
      const uint4 v = *reinterpret_cast<const uint4*>(cache + i);
      f(v.x, i);
      f(v.y, i + 1);
      f(v.z, i + 2);
      f(v.w, i + 3);
    }
    for (int32_t i = max(a4, b4) + me; i < to; i += threads) f(key_at(i), i);
  };
  uint32_t prefix = 0, left = (uint32_t)need;  // the digits found so far; the rank among what is left
  int done = 32 - __clz(high - low);           // bits of the distance not yet looked at
  uint32_t in_bin = (uint32_t)(hi - lo);       // keys that share the digits found so far
  int pass = 0;
  for (; done > 0 && in_bin > kSelExchange; ++pass) {
    const int shift = max(0, done - 11);
    const uint32_t mask = (1u << (done - shift)) - 1u, span = 0xFFFFFFFFu >> (32 - done);
    uint32_t* hist = sh.hist[pass & 1];
    each_key(i_lo, n, tid, kSelThreads, [&](uint32_t k, int32_t) {
      const uint32_t x = k - low;
      if (x - prefix <= span) atomicAdd(&hist[(x >> shift) & mask], 1u);
    });
    __syncthreads();
    for (int c = warp; c < kCoarse; c += kSelWarps) {
      const uint32_t v = __reduce_add_sync(0xffffffffu, hist[64 * c + lane] + hist[64 * c + 32 + lane]);
      if (lane == 0) sh.coarse[pass & 1][c] = v;
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    // the coarse bin of the left-th largest key: bins from the top down, lane l takes bin 31 - l
    {
      const uint32_t r = tid / kCoarse, c = tid % kCoarse;
      sh.all[r][c] = r < C ? cluster_load(cluster_peer(smem_u32(&sh.coarse[pass & 1][c]), r)) : 0u;
    }
    __syncthreads();
    if (warp == 0) {
      uint32_t mine = 0;
      for (uint32_t r = 0; r < C; ++r) mine += sh.all[r][kCoarse - 1 - lane];
      uint32_t sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      if (sum - mine < left && left <= sum) {
        sh.digit = kCoarse - 1 - lane;
        sh.above = sum - mine;
      }
    }
    __syncthreads();
    const uint32_t coarse = sh.digit;
    const uint32_t left_in = left - sh.above;
    for (uint32_t r = tid / 64; r < C; r += kSelThreads / 64)
      sh.all[r][tid % 64] = cluster_load(cluster_peer(smem_u32(hist + 64 * coarse + tid % 64), r));
    __syncthreads();
    if (warp == 0) {  // lane l takes bins 63 - 2 l and 62 - 2 l of the 64
      uint32_t a = 0, b = 0;
      for (uint32_t r = 0; r < C; ++r) {
        a += sh.all[r][63 - 2 * lane];
        b += sh.all[r][62 - 2 * lane];
      }
      uint32_t sum = a + b;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      const uint32_t before = sum - a - b;
      if (before < left_in && left_in <= sum) {
        const bool top = left_in <= before + a;
        sh.digit = 64 * coarse + 62 - 2 * lane + (top ? 1 : 0);
        sh.above = top ? before : before + a;
        sh.in_bin = top ? a : b;
      }
    }
    __syncthreads();
    const uint32_t digit = sh.digit;
    prefix |= digit << shift;
    left = left_in - sh.above;
    in_bin = sh.in_bin;
    done = shift;
    // this CTA's keys above the digit
    uint32_t mine = 0;
    for (uint32_t c = digit + 1 + tid; c < kBins; c += kSelThreads) mine += hist[c];
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0 && mine > 0) atomicAdd(&sh.over, mine);
    // the other histogram, which the peers last read before this pass's meeting, is for the next
    // pass or the exchange
    for (int i = tid; i < kBins; i += kSelThreads) sh.hist[(pass + 1) & 1][i] = 0;
    __syncthreads();
  }

  // Exchange the keys that share the digits; when there are no more bits they are all equal, and
  // only their number is needed. Each warp goes over its part of the slice and counts the keys above
  // the digits on the way.
  uint32_t* list = sh.hist[pass & 1];
  const uint32_t span = done > 0 ? 0xFFFFFFFFu >> (32 - done) : 0u, top = prefix + span;
  const int32_t part = (int32_t)((((int64_t)n + kSelWarps - 1) / kSelWarps + 127) & ~127);
  const int32_t i_begin = max(i_lo, min(n, warp * part));
  const int32_t i_end = max(i_begin, min(n, (warp + 1) * part));
  {
    int32_t above = 0, equal = 0;
    each_key(i_begin, i_end, lane, 32, [&](uint32_t k, int32_t i) {
      const uint32_t x = k - low;
      above += x > top;
      if (x - prefix <= span) {
        ++equal;
        if (done > 0) {
          const uint32_t at = atomicAdd(&sh.listed, 1u);
          list[at] = x;
          sh.list_at[at] = i;
        }
      }
    });
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
      sh.warp_over[warp] = above;
      sh.warp_tied[warp] = done > 0 ? 0 : equal;
      if (done == 0 && equal > 0) atomicAdd(&sh.listed, (uint32_t)equal);
    }
  }
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  uint32_t over_r = 0, listed_r = 0;  // of CTA `lane`
  if (lane < C) {
    over_r = cluster_load(cluster_peer(smem_u32(&sh.over), lane));
    listed_r = cluster_load(cluster_peer(smem_u32(&sh.listed), lane));
  }
  int32_t over = (int32_t)__reduce_add_sync(0xffffffffu, lane < rank ? over_r : 0u);
  int32_t tied = (int32_t)__reduce_add_sync(0xffffffffu, lane < rank ? listed_r : 0u);
  if (done > 0) {
    uint32_t upto = listed_r;  // inclusive scan over the CTAs
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    // all lists, CTA after CTA, in the place of the histogram read before the last meeting
    uint32_t* got = sh.hist[(pass + 1) & 1];
    for (uint32_t r = warp; r < C; r += kSelWarps) {
      const uint32_t size = __shfl_sync(0xffffffffu, listed_r, r);
      const uint32_t at = __shfl_sync(0xffffffffu, upto, r) - size;
      for (uint32_t i = lane; i < size; i += 32)
        got[at + i] = cluster_load(cluster_peer(smem_u32(list + i), r));
    }
    __syncthreads();
    const uint32_t mine_from = (uint32_t)tied;
    uint32_t x[kSelRounds];
    bool real[kSelRounds];
#pragma unroll
    for (int u = 0; u < kSelRounds; ++u) {
      real[u] = (uint32_t)(tid + u * kSelThreads) < in_bin;
      x[u] = real[u] ? got[tid + u * kSelThreads] : 0u;
    }
    for (int round = 0; done > 0; ++round) {
      const int shift = max(0, done - 7);
      const uint32_t mask = (1u << (done - shift)) - 1u, among = 0xFFFFFFFFu >> (32 - done);
      uint32_t* bins = sh.bins7[round & 1];
#pragma unroll
      for (int u = 0; u < kSelRounds; ++u)
        if (real[u] && x[u] - prefix <= among) atomicAdd(&bins[(x[u] >> shift) & mask], 1u);
      __syncthreads();
      // every warp finds the digit; lane l takes bins 124 - 4 l .. 127 - 4 l
      const uint4 v = *reinterpret_cast<const uint4*>(bins + 124 - 4 * lane);
      const uint32_t mine = v.x + v.y + v.z + v.w;
      uint32_t sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      uint32_t before = sum - mine, digit = (uint32_t)(127 - 4 * lane), share = v.w;
      const bool here = before < left && left <= sum;
      if (before + v.w < left) {
        before += v.w;
        --digit;
        share = v.z;
        if (before + v.z < left) {
          before += v.z;
          --digit;
          share = v.y;
          if (before + v.y < left) {
            before += v.y;
            --digit;
            share = v.x;
          }
        }
      }
      const int src = __ffs((int)__ballot_sync(0xffffffffu, here)) - 1;
      prefix |= __shfl_sync(0xffffffffu, digit, src) << shift;
      left -= __shfl_sync(0xffffffffu, before, src);
      done = shift;
      if (done > 0 && __shfl_sync(0xffffffffu, share, src) == 1u) {
        // one key is left: it is the edge (as a rule the case after one round or two)
        const uint32_t rest = 0xFFFFFFFFu >> (32 - done);
#pragma unroll
        for (int u = 0; u < kSelRounds; ++u)
          if (real[u] && x[u] - prefix <= rest) sh.digit = x[u];
        __syncthreads();
        prefix = sh.digit;
        break;
      }
      // the other bins: every warp read them before the barrier above
      if (tid < 128) sh.bins7[(round + 1) & 1][tid] = 0;
      __syncthreads();
    }
    // how many of the lists of the CTAs before this one are kept, or equal the threshold
    int32_t more = 0, equal = 0;
#pragma unroll
    for (int u = 0; u < kSelRounds; ++u) {
      const bool theirs = (uint32_t)(tid + u * kSelThreads) < mine_from;
      more += __syncthreads_count(theirs && x[u] > prefix);
      equal += __syncthreads_count(theirs && x[u] == prefix);
    }
    over += more;
    tied = equal;
    // this CTA's exchanged keys, now that the edge is known, to the warps' counts
    const int32_t listed = (int32_t)sh.listed;
    for (int32_t i = tid; i < listed; i += kSelThreads) {
      const uint32_t v = list[i];
      if (v > prefix) atomicAdd(&sh.warp_over[sh.list_at[i] / part], 1);
      else if (v == prefix) atomicAdd(&sh.warp_tied[sh.list_at[i] / part], 1);
    }
    __syncthreads();
  }
  cluster_arrive();  // awaited at the end: a CTA's shared memory stays while peers read it

  // keys above `edge` are kept, and the first `left` of those equal to it
  const uint32_t edge = low + prefix;
  const int32_t my_tied = sh.warp_tied[warp];
  over += __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_over[lane] : 0);
  tied += __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_tied[lane] : 0);
  const uint32_t below = (1u << lane) - 1u;
  // keys equal to the edge: a part before the left-th of them keeps them all, one behind it none
  // (written as comparisons: of int32 a, b and q = max(0, min(a, b)), nvcc 13.0.88 compiles q == b to
  // false where it holds, as a kernel of that line alone shows, unless ptxas runs at -O0; q is right)
  const int32_t to_come = (int32_t)left - tied;
  const int32_t quota = to_come <= 0 ? 0 : to_come < my_tied ? to_come : my_tied;
  int32_t* dst = out + lo + over + (to_come > 0 ? tied : (int32_t)left);
  if ((quota == 0 || quota == my_tied) && (i_begin & 3) == 0 && (i_end & 3) == 0 && i_end <= cached) {
    // 128 keys at a time, four neighbours per lane (no key is as large as 2^32 - 1: edge + 1 exists)
    const uint32_t least = quota == my_tied ? edge : edge + 1u;
#pragma unroll 2
    for (int32_t i0 = i_begin; i0 < i_end; i0 += 128) {
      const int32_t i = i0 + 4 * lane;
      const bool real = i < i_end;
      const uint4 v = real ? *reinterpret_cast<const uint4*>(cache + i) : make_uint4(0u, 0u, 0u, 0u);
      const bool take[4] = {real && v.x >= least, real && v.y >= least, real && v.z >= least,
                            real && v.w >= least};
      int32_t* d = dst;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t m = __ballot_sync(0xffffffffu, take[e]);
        d += __popc(m & below);
        dst += __popc(m);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (take[e]) *d++ = t0 + i + e;
      }
    }
  } else {
    int32_t rank_tied = 0;
    for (int32_t i0 = i_begin; i0 < i_end; i0 += 32) {
      const int32_t i = i0 + lane;
      const bool real = i < i_end;
      const uint32_t k = real ? key_at(i) : 0u;
      const uint32_t m_tied = __ballot_sync(0xffffffffu, real && k == edge);
      const bool take =
          real && (k > edge || (k == edge && rank_tied + __popc(m_tied & below) < quota));
      const uint32_t m = __ballot_sync(0xffffffffu, take);
      if (take) dst[__popc(m & below)] = t0 + i;
      dst += __popc(m);
      rank_tied += __popc(m_tied);
    }
  }
  for (int64_t j = first; j < lo; j += step) out[j] = (int32_t)j;
  for (int64_t j = first; j < len - hi; j += step) out[lo + need + j] = (int32_t)(hi + j);
  cluster_wait();
}

struct CompactParams {
  const int32_t* index;    // [num_seqs][Hkv or 1][index_stride]
  int64_t index_stride;
  int32_t per_head;
  const int32_t* seq_lens;
  const int32_t* keep;
  const int32_t* block_table;
  const int32_t* dst_table;
  int32_t max_pages, dst_max_pages, num_pages;
  uint8_t* pool;
  float* weights;          // [num_seqs][Hkv][w_stride], or null
  int64_t w_stride;
  int32_t Hkv;
  int32_t* status;
};

// One cluster per (sequence, KV head, part): the K rows, the V rows, the weights; or, with few sequences
// and heads, two clusters for the K and two for the V rows, each with two of the four 16-byte pieces
// of a row's codes and one of its two words of scales (bytes that no other part touches). The cluster
// takes its rows in waves: in a wave every thread loads what it moves into registers (a piece of the
// codes, and for half of the threads four scales, of kMoveRows rows), the cluster meets, and the wave
// is stored. The next wave's reads, which lie behind the wave's rows, are on their way meanwhile.
//
// Bounds: 296 bytes per kept row and KV head, but the rows lie apart: a K row's codes are four
// 16-byte pieces in sectors that hold a neighbour's piece as well, its scales two words in two more,
// and DRAM gives 64 bytes at a time. 4 x 4 sets, 16384 kept of 131072: 78 MB of rows move, 184 MB
// cross the memory bus, in 43 us (4.3 TB/s). One CTA per part took 272 us, waves with branches
// around the loads (and 144 bytes of spills) 74 us, unconditional loads without reads ahead 45 us (8
// bytes; 20 now, and none in halves), eight rows per thread at two CTAs per SM 59 us, two rows at six 55 us, clusters of nine
// instead of eight (432 CTAs, not 384) the same 43. A gather of the same K and V rows into another
// buffer, without any order or meeting, takes 37 us whatever its grid.
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;                                // rows in flight per thread
constexpr int kMoveMaxCluster = 16;
constexpr int kMoveCtasPerSm = 3;
// rows of a CTA per wave, codes and scales, when a part has kPieces of a row's pieces
template <int kPieces>
constexpr int kMoveTile = kMoveThreads / kPieces * kMoveRows;

template <int kPieces>
__global__ void __launch_bounds__(kMoveThreads, kMoveCtasPerSm) compact_kernel(const CompactParams p) {
  const uint32_t C = cluster_size(), rank = cluster_rank();
  constexpr int kSplit = 4 / kPieces, kTile = kMoveTile<kPieces>;
  const int parts = 2 * kSplit + (p.weights != nullptr ? 1 : 0);
  const int64_t unit = blockIdx.x / C;
  const int part = (int)(unit % parts), head = (int)(unit / parts % p.Hkv);
  const int64_t seq = unit / parts / p.Hkv;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // e.g. for the selection's index
  const int32_t len = p.seq_lens[seq], keep = p.keep[seq];
  const int32_t kept = min(len, keep);
  // the same for every CTA of the cluster
  if (len < 0 || keep < 0 || kept > p.index_stride || len > (int64_t)p.max_pages * kPage ||
      kept > (int64_t)p.dst_max_pages * kPage || (p.weights != nullptr && len > p.w_stride)) {
    if (tid == 0 && rank == 0) flag_status(p.status, KV_NVFP4_DEV_BAD_POS);
    return;
  }
  const int32_t* index =
      p.index + (seq * (p.per_head ? p.Hkv : 1) + (p.per_head ? head : 0)) * p.index_stride;
  if (part == 2 * kSplit) {
    float* w = p.weights + (seq * p.Hkv + head) * p.w_stride;
    const int64_t wave = (int64_t)C * kMoveThreads * kMoveRows;
    for (int64_t j0 = 0; j0 < kept; j0 += wave) {
      const int64_t first = j0 + (int64_t)rank * (kMoveThreads * kMoveRows) + tid;
      int32_t t[kMoveRows];
      float v[kMoveRows];
#pragma unroll
      for (int u = 0; u < kMoveRows; ++u)
        t[u] = first + u * kMoveThreads < kept ? index[first + u * kMoveThreads] : 0;
#pragma unroll
      for (int u = 0; u < kMoveRows; ++u) {
        const bool ok = t[u] >= 0 && t[u] < len;
        if (!ok) flag_status(p.status, KV_NVFP4_DEV_BAD_POS);
        v[u] = ok && first + u * kMoveThreads < kept ? w[t[u]] : 0.f;
        if (!ok) t[u] = -1;
      }
      cluster_arrive();
      cluster_wait();
#pragma unroll
      for (int u = 0; u < kMoveRows; ++u)
        if (t[u] >= 0 && first + u * kMoveThreads < kept) w[first + u * kMoveThreads] = v[u];
    }
    // every read lies before the last meeting
    for (int64_t j = kept + (int64_t)rank * kMoveThreads + tid; j < len; j += (int64_t)C * kMoveThreads)
      w[j] = 0.f;
    return;
  }
  const int32_t* src_table = p.block_table + seq * p.max_pages;
  const int32_t* dst_table = p.dst_table + seq * p.dst_max_pages;
  const int64_t block = (int64_t)p.Hkv * 9216;
  const bool keys = part < kSplit;
  const int half = part % kSplit, piece = half * kPieces + tid % kPieces;
  const int word = kSplit == 1 ? piece & 1 : half;
  const bool with_scales = kSplit == 1 ? piece < 2 : tid % kPieces == 0;
  // byte offsets of this thread's 16 code bytes and four scales of a slot
  auto code_at = [&](int slot) {
    return keys ? head * 4096 + (slot >> 3) * 512 + piece * 128 + (slot & 7) * 16
                : p.Hkv * 4608 + head * 4096 + slot * 64 + piece * 16;
  };
  auto scale_at = [&](int slot) {
    return keys ? kscale_offset(p.Hkv, head, slot, word)
                : p.Hkv * 8704 + head * 512 + slot * 8 + 4 * word;
  };
  const int64_t wave = (int64_t)C * kTile;
  constexpr int kApart = kMoveThreads / kPieces;  // rows between a thread's rows
  const int64_t first = (int64_t)rank * kTile + tid / kPieces;
  int32_t bad = 0;
  struct Rows {
    uint4 c[kMoveRows];
    uint32_t sc[kMoveRows];
    int32_t to[kMoveRows];
  };
  int32_t t[kMoveRows], from[kMoveRows];  // of the wave that is loaded next
  auto find = [&](int64_t j) {             // its old slots and pages
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) t[u] = j + u * kApart < kept ? index[j + u * kApart] : -1;
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const bool real = j + u * kApart < kept, ok = t[u] >= 0 && t[u] < len;
      if (real && !ok) bad |= KV_NVFP4_DEV_BAD_POS;
      if (!ok) t[u] = -1;
      from[u] = ok ? src_table[t[u] / kPage] : -1;
    }
  };
  auto load = [&](int64_t j, Rows& r) {
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) r.to[u] = t[u] >= 0 ? dst_table[(j + u * kApart) / kPage] : -1;
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const bool ok = from[u] >= 0 && from[u] < p.num_pages && r.to[u] >= 0 && r.to[u] < p.num_pages;
      if (t[u] >= 0 && !ok) bad |= KV_NVFP4_DEV_BAD_PAGE;
      // a row that is already there stays; it and a skipped one read slot 0 of page 0 for nothing
      const bool move = ok && (t[u] != j + u * kApart || from[u] != r.to[u]);
      const uint8_t* src = p.pool + (move ? from[u] * block : 0);
      const int slot = move ? t[u] % kPage : 0;
      r.c[u] = *reinterpret_cast<const uint4*>(src + code_at(slot));
      r.sc[u] = *reinterpret_cast<const uint32_t*>(src + scale_at(slot));
      if (!move) r.to[u] = -1;
    }
  };
  auto store = [&](int64_t j, const Rows& r) {
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      if (r.to[u] < 0) continue;
      const int slot = (int)((j + u * kApart) % kPage);
      uint8_t* dst = p.pool + r.to[u] * block;
      *reinterpret_cast<uint4*>(dst + code_at(slot)) = r.c[u];
      if (with_scales) *reinterpret_cast<uint32_t*>(dst + scale_at(slot)) = r.sc[u];
    }
  };
  Rows a, b;
  if (kept > 0) {
    find(first);
    load(first, a);
    find(first + wave);
  }
  for (int64_t j0 = 0; j0 < kept; j0 += 2 * wave) {
    // the wave is read whole before any of its rows is written; the next one's reads (of slots
    // behind the wave) start while the cluster meets
    cluster_arrive();
    if (j0 + wave < kept) {
      load(first + j0 + wave, b);
      find(first + j0 + 2 * wave);
    }
    cluster_wait();
    store(first + j0, a);
    if (j0 + wave >= kept) break;
    cluster_arrive();
    if (j0 + 2 * wave < kept) {
      load(first + j0 + 2 * wave, a);
      find(first + j0 + 3 * wave);
    }
    cluster_wait();
    store(first + j0 + wave, b);
  }
  if (bad != 0) flag_status(p.status, bad);
}

// The largest cluster, a power of two up to `most`, of which the current device can place one.
int largest_cluster(const void* kernel, int threads, size_t smem, int most) {
  for (int C = most; C > 1; C /= 2) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0) return C;
    cudaGetLastError();  // too large a cluster is no launch error: do not leave it set
  }
  return 1;
}

}  // namespace

cudaError_t launch_evict_select(const float* weights, int64_t w_stride, const int32_t* seq_lens,
                                const int32_t* keep, int32_t num_seqs, int32_t per_head,
                                int32_t sink, int32_t recent, int32_t* index, int64_t index_stride,
                                int32_t Hkv, int32_t num_sms, int32_t* status,
                                cudaStream_t stream) {
  static int of_device[64] = {};  // clusters of CTAs with all of the shared memory
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  int largest = dev >= 0 && dev < 64 ? of_device[dev] : 0;
  if (largest == 0) {
    for (const void* kf : {(const void*)select_kernel<false>, (const void*)select_kernel<true>}) {
      cudaError_t e = cudaFuncSetAttribute(kf, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)sizeof(SelectShared) + 4 * kSelMaxCached);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kf, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    largest = largest_cluster((const void*)select_kernel<true>, kSelThreads,
                              sizeof(SelectShared) + 4 * kSelMaxCached, kSelMaxCluster);
    if (dev >= 0 && dev < 64) of_device[dev] = largest;
  }
  // The lengths are on the device, so the cluster is sized for the longest that the accounts hold:
  // as few CTAs as keep the keys in shared memory, and up to eight while SMs are left and a CTA has
  // 2048 keys. Measured (us, before the programmatic launch, C = 1, 2, 4, 8, 16): 4 sets of 4000 slots 12.3, 10.3, 10.3, 10.3, 14.4;
  // 4 of 20000 16.4, 14.4, 12.3, 12.3, 14.4; 8 of 131072 (from C = 4) 22.6, 18.4, 22.6; 16 of 131072
  // 22.6, 22.6, 35; 48 of 40000 24.6, 18.4, 18.5, 28, 62; 128 of 4000 12.3, 12.7, 22, 43, 137.
  const int64_t sets = (int64_t)num_seqs * (per_head ? Hkv : 1);
  int64_t C = 1;
  while (C < largest &&
         (C * kSelMaxCached < w_stride || (C < 8 && sets * C * 2 <= num_sms && C * 2048 < w_stride)))
    C *= 2;
  const int64_t slice = (w_stride + C - 1) / C + 64;
  const int64_t cached = slice < kSelMaxCached ? slice : kSelMaxCached;
  const SelectParams p{weights, w_stride, seq_lens, keep,   index,           index_stride,
                       Hkv,     per_head, sink,     recent, (int32_t)cached, status};
  const int64_t grid = sets * C;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = sizeof(SelectShared) + 4 * (size_t)cached;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const bool vec = w_stride % 4 == 0 && (reinterpret_cast<uintptr_t>(weights) & 15u) == 0;
  return vec ? cudaLaunchKernelEx(&cfg, select_kernel<true>, p)
             : cudaLaunchKernelEx(&cfg, select_kernel<false>, p);
}

cudaError_t launch_evict_compact(const int32_t* index, int64_t index_stride, int32_t per_head,
                                 const int32_t* seq_lens, const int32_t* keep, int32_t num_seqs,
                                 const int32_t* block_table, int32_t max_pages, int32_t num_pages,
                                 uint8_t* pool, const int32_t* dst_table, int32_t dst_max_pages,
                                 float* weights, int64_t w_stride, int32_t Hkv, int32_t num_sms,
                                 int32_t* status, cudaStream_t stream) {
  const CompactParams p{index,     index_stride,  per_head,  seq_lens, keep,    block_table,
                        dst_table, max_pages,     dst_max_pages, num_pages, pool, weights,
                        w_stride,  Hkv,           status};
  static int of_device[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  int largest = dev >= 0 && dev < 64 ? of_device[dev] : 0;
  if (largest == 0) {
    for (const void* kf : {(const void*)compact_kernel<4>, (const void*)compact_kernel<2>}) {
      const cudaError_t e =
          cudaFuncSetAttribute(kf, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    largest = largest_cluster((const void*)compact_kernel<4>, kMoveThreads, 0, kMoveMaxCluster);
    if (dev >= 0 && dev < 64) of_device[dev] = largest;
  }
  // the kept counts are on the device: sized for the most that the index holds, a wave per CTA, and
  // no more CTAs than run at once; in halves when clusters of the most CTAs still find places. One
  // sequence, four heads, 16384 kept of 131072: 22.7 us with clusters of 8, 14.6 of 16, 9.9 in halves;
  // two heads, 60000 of 600000: 88.9, 46.8, 29.2; one head, 5000 of 20000: 7.2 of 16, 6.6 in halves
  const int64_t places = kMoveCtasPerSm * (int64_t)num_sms, pairs = (int64_t)num_seqs * Hkv;
  const int extra = weights != nullptr ? 1 : 0;
  const bool halves = pairs * (4 + extra) * kMoveMaxCluster <= places;
  const int64_t units = pairs * ((halves ? 4 : 2) + extra);
  const int64_t tile = halves ? kMoveTile<2> : kMoveTile<4>;
  int64_t C = 1;
  while (C < largest && C * tile < index_stride && units * C * 2 <= places) C *= 2;
  if (units * C > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return halves ? cudaLaunchKernelEx(&cfg, compact_kernel<2>, p)
                : cudaLaunchKernelEx(&cfg, compact_kernel<4>, p);
}

}  // namespace kvnvfp4
