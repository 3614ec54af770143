// Eviction from the paged cache by accumulated attention weight: the choice of the slots to keep
// (kv_nvfp4_evict_select) and the compaction of the cache to them (kv_nvfp4_evict_compact).
//
// Select. Per set of slots (a KV head's, or a sequence's when all heads share one set) the slots
// [0, sink) and [len - recent, len) come first, then the rest by weight, ties to the lowest slot;
// the first min(len, keep) of that order are listed in ascending slot order. The weights are mapped
// to unsigned keys of the same order (NaN to 0, below every value) and the smallest kept key is
// found by a radix select, eight bits at a time.
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

constexpr int kSelThreads = 1024;

__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_digit, s_need;
  __shared__ int32_t warp_kept[32], warp_tied[32];
  const int sets = p.per_head ? p.Hkv : 1;
  const int seq = blockIdx.x / sets, set = blockIdx.x % sets;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t len = p.seq_lens[seq], keep = p.keep[seq];
  const int32_t kept = min(len, keep);
  if (len < 0 || keep < 0 || len > p.w_stride || kept > p.index_stride) {
    if (tid == 0) flag_status(p.status, KV_NVFP4_DEV_BAD_POS);
    return;
  }
  int32_t* out = p.index + ((int64_t)seq * sets + set) * p.index_stride;
  const float* w = p.weights + ((int64_t)seq * p.Hkv + set) * p.w_stride;
  const int heads = p.per_head ? 1 : p.Hkv;
  // [lo, hi): the slots that are not protected
  const int32_t lo = min(len, p.sink), hi = max(lo, p.recent < len ? len - p.recent : 0);
  if (kept == len || lo + (len - hi) >= kept) {  // no choice by weight: the first kept of them
    for (int32_t j = tid; j < kept; j += kSelThreads)
      out[j] = kept == len || j < lo ? j : hi + (j - lo);
    return;
  }
  const int32_t need = kept - lo - (len - hi);  // 1 <= need < hi - lo
  // radix select: `prefix` holds the digits found so far of the need-th largest key
  uint32_t prefix = 0, left = (uint32_t)need;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int32_t t = lo + tid; t < hi; t += kSelThreads) {
      const uint32_t k = order_key(set_weight(w, p.w_stride, heads, t));
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t above = 0;
      int d = 255;
      while (d > 0 && above + hist[d] < left) above += hist[d--];
      s_digit = (uint32_t)d;
      s_need = left - above;
    }
    __syncthreads();
    prefix |= s_digit << shift;
    left = s_need;
    __syncthreads();
  }
  // keys above `prefix` are kept, and the first `left` of those equal to it
  for (int32_t j = tid; j < lo; j += kSelThreads) out[j] = j;
  for (int32_t j = tid; j < len - hi; j += kSelThreads) out[lo + need + j] = hi + j;
  int32_t n_kept = 0, n_tied = 0;  // so far, over all threads
  for (int32_t t0 = lo; t0 < hi; t0 += kSelThreads) {
    const int32_t t = t0 + tid;
    uint32_t k = 0;
    if (t < hi) k = order_key(set_weight(w, p.w_stride, heads, t));
    const bool over = t < hi && k > prefix, tied = t < hi && k == prefix;
    const uint32_t m_over = __ballot_sync(0xffffffffu, over);
    const uint32_t m_tied = __ballot_sync(0xffffffffu, tied);
    if (lane == 0) {
      warp_kept[warp] = __popc(m_over);
      warp_tied[warp] = __popc(m_tied);
    }
    __syncthreads();
    int32_t over_before = 0, tied_before = 0, all_over = 0, all_tied = 0;
    for (int i = 0; i < 32; ++i) {
      if (i < warp) {
        over_before += warp_kept[i];
        tied_before += warp_tied[i];
      }
      all_over += warp_kept[i];
      all_tied += warp_tied[i];
    }
    const uint32_t below = (1u << lane) - 1u;
    over_before += n_kept + __popc(m_over & below);
    tied_before += n_tied + __popc(m_tied & below);
    if (over || (tied && tied_before < (int32_t)left))
      out[lo + over_before + min(tied_before, (int32_t)left)] = t;
    n_kept += all_over;
    n_tied += all_tied;
    __syncthreads();
  }
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

constexpr int kMoveThreads = 256;

// One CTA per (sequence, KV head, part): part 0 the K rows, 1 the V rows, 2 the weights. Rows in
// tiles of 64, four threads per row.
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const CompactParams p) {
  const int parts = p.weights != nullptr ? 3 : 2;
  const int part = blockIdx.x % parts, head = blockIdx.x / parts % p.Hkv;
  const int seq = blockIdx.x / parts / p.Hkv;
  const int tid = threadIdx.x;
  const int32_t len = p.seq_lens[seq], keep = p.keep[seq];
  const int32_t kept = min(len, keep);
  if (len < 0 || keep < 0 || kept > p.index_stride || len > (int64_t)p.max_pages * kPage ||
      kept > (int64_t)p.dst_max_pages * kPage || (part == 2 && len > p.w_stride)) {
    if (tid == 0) flag_status(p.status, KV_NVFP4_DEV_BAD_POS);
    return;
  }
  const int32_t* index =
      p.index + ((int64_t)seq * (p.per_head ? p.Hkv : 1) + (p.per_head ? head : 0)) * p.index_stride;
  if (part == 2) {
    float* w = p.weights + ((int64_t)seq * p.Hkv + head) * p.w_stride;
    for (int32_t j0 = 0; j0 < kept; j0 += kMoveThreads) {
      const int32_t j = j0 + tid;
      float v = 0.f;
      bool ok = false;
      if (j < kept) {
        const int32_t t = index[j];
        ok = t >= 0 && t < len;
        if (ok) v = w[t];
        else flag_status(p.status, KV_NVFP4_DEV_BAD_POS);
      }
      __syncthreads();
      if (ok) w[j] = v;
    }
    __syncthreads();
    for (int32_t j = kept + tid; j < len; j += kMoveThreads) w[j] = 0.f;
    return;
  }
  const int32_t* src_table = p.block_table + (int64_t)seq * p.max_pages;
  const int32_t* dst_table = p.dst_table + (int64_t)seq * p.dst_max_pages;
  const int64_t block = (int64_t)p.Hkv * 9216;
  const int row = tid >> 2, piece = tid & 3;
  // byte offsets of this thread's 16 code bytes and (pieces 0, 1) four scales of a slot
  auto code_at = [&](int slot) {
    return part == 0 ? head * 4096 + (slot >> 3) * 512 + piece * 128 + (slot & 7) * 16
                     : p.Hkv * 4608 + head * 4096 + slot * 64 + piece * 16;
  };
  auto scale_at = [&](int slot) {
    return part == 0 ? kscale_offset(p.Hkv, head, slot, piece & 1)
                     : p.Hkv * 8704 + head * 512 + slot * 8 + 4 * (piece & 1);
  };
  for (int32_t j0 = 0; j0 < kept; j0 += kPage) {
    const int32_t j = j0 + row;
    uint8_t* dst = nullptr;
    uint4 c = make_uint4(0u, 0u, 0u, 0u);
    uint32_t sc = 0;
    if (j < kept) {
      const int32_t t = index[j];
      const int32_t to = dst_table[j / kPage];
      if (t < 0 || t >= len) {
        flag_status(p.status, KV_NVFP4_DEV_BAD_POS);
      } else {
        const int32_t from = src_table[t / kPage];
        if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
          flag_status(p.status, KV_NVFP4_DEV_BAD_PAGE);
        } else {
          const uint8_t* src = p.pool + from * block;
          c = *reinterpret_cast<const uint4*>(src + code_at(t % kPage));
          if (piece < 2) sc = *reinterpret_cast<const uint32_t*>(src + scale_at(t % kPage));
          dst = p.pool + to * block;
        }
      }
    }
    __syncthreads();  // the tile is read whole before any of its rows is written
    if (dst != nullptr) {
      *reinterpret_cast<uint4*>(dst + code_at(row)) = c;
      if (piece < 2) *reinterpret_cast<uint32_t*>(dst + scale_at(row)) = sc;
    }
  }
}

}  // namespace

cudaError_t launch_evict_select(const float* weights, int64_t w_stride, const int32_t* seq_lens,
                                const int32_t* keep, int32_t num_seqs, int32_t per_head,
                                int32_t sink, int32_t recent, int32_t* index, int64_t index_stride,
                                int32_t Hkv, int32_t* status, cudaStream_t stream) {
  const SelectParams p{weights, w_stride, seq_lens, keep, index, index_stride,
                       Hkv,     per_head, sink,     recent, status};
  const int64_t sets = (int64_t)num_seqs * (per_head ? Hkv : 1);
  if (sets > 0x7FFFFFFF) return cudaErrorInvalidValue;
  select_kernel<<<(unsigned)sets, kSelThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_evict_compact(const int32_t* index, int64_t index_stride, int32_t per_head,
                                 const int32_t* seq_lens, const int32_t* keep, int32_t num_seqs,
                                 const int32_t* block_table, int32_t max_pages, int32_t num_pages,
                                 uint8_t* pool, const int32_t* dst_table, int32_t dst_max_pages,
                                 float* weights, int64_t w_stride, int32_t Hkv, int32_t* status,
                                 cudaStream_t stream) {
  const CompactParams p{index,     index_stride,  per_head,  seq_lens, keep,    block_table,
                        dst_table, max_pages,     dst_max_pages, num_pages, pool, weights,
                        w_stride,  Hkv,           status};
  const int64_t grid = (int64_t)num_seqs * Hkv * (weights != nullptr ? 3 : 2);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  compact_kernel<<<(unsigned)grid, kMoveThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace kvnvfp4
