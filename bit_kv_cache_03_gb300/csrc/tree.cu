// Trees of drafted tokens around their attention (kv_nvfp4_tree_attn, in decode.cu and tile.cu): the
// masks, slots and positions of a tree's nodes (kv_nvfp4_tree_mask), and after the model has answered
// the path that it agrees with, its rows moved behind the cache (kv_nvfp4_tree_accept).
//
// No counterpart in the pages, which verify a chain of drafts.

#include <cstdint>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"

namespace kvnvfp4 {

namespace {

constexpr int kMaxNodes = KV_NVFP4_MAX_TREE;
constexpr int kMaxWords = kMaxNodes / 32;
constexpr int kTreePages = kMaxNodes / kPage + 1;  // pages that a tree's slots can touch

// The accounts that the block table is under (refs null: none).
struct Accounts {
  const int32_t* block_table;  // [.][max_pages]
  const int32_t* refs;         // [num_pages]
  int32_t max_pages, num_pages;
};

// Whether the j-th page from the one of slot `base` on is another sequence's as well and takes one of n
// slots from there.
__device__ __forceinline__ bool shared_page(const Accounts& a, int64_t seq, int32_t base, int n, int j) {
  const int64_t place = base / kPage + j;
  if (place * kPage >= (int64_t)base + n || place >= a.max_pages) return false;
  const int32_t page = a.block_table[seq * a.max_pages + place];
  return page >= 0 && page < a.num_pages && a.refs[page] > 1;
}

struct TreeMaskParams {
  const int32_t* parents;    // [num_seqs][n]
  const int32_t* lens;       // [num_seqs] slots before the tree
  const int32_t* first_pos;  // [num_seqs], or null: lens
  uint32_t* mask;            // [num_seqs][n][W]
  int32_t* seq_ids;          // [num_seqs * n], as the next two, or all null
  int32_t* slots;
  int32_t* positions;
  Accounts accounts;
  int32_t n;
  int32_t* status;
};

// One CTA per tree, one thread per node. The set of a node is its own bit and its parent's set; with
// every node holding the set of its nearest 2^r levels and a pointer to the one above them, one step
// joins the two and doubles the levels: log2 of the depth steps in the place of one per level. A
// pointer ends at the cache (-1) or, for a node that hangs nowhere, at -2, whose set is empty.
//
// Bounds: the launch, and log2 of the depth pairs of barriers. Replayed from a graph a tree of 8 takes
// 1.3 to 1.5 us, 128 trees of 256 (1.4 MB written, 0.2 us of HBM time) 3.2 to 3.4, each 0.3 more with
// accounts (two dependent loads beside the first steps); called, both take the host's 5.3.
template <int kWords>
__global__ void __launch_bounds__(32 * kWords) tree_mask_kernel(const TreeMaskParams p) {
  __shared__ uint32_t sets[kWords][32 * kWords];
  __shared__ int32_t above[32 * kWords];
  const int i = threadIdx.x, n = p.n, W = (n + 31) >> 5;  // W <= kWords: every node has its thread
  const int64_t seq = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int32_t len = p.lens[seq];
  const int32_t first = p.first_pos != nullptr ? p.first_pos[seq] : len;
  int32_t up = i < n ? p.parents[seq * n + i] : -2;
  auto no_place = [&]() {  // what an earlier call left there would be appended again
    if (p.slots != nullptr && i < n)
      p.seq_ids[seq * n + i] = p.slots[seq * n + i] = p.positions[seq * n + i] = -1;
  };
  if (len < 0 || first < 0 || len > 0x7FFFFFFF - n || first > 0x7FFFFFFF - n) {  // for the whole CTA
    if (i == 0) flag_status(p.status, KV_NVFP4_DEV_BAD_POS);
    no_place();
    return;
  }
  // (a thread per page: there are at least 32)
  const bool shared = p.accounts.refs != nullptr && i < kTreePages &&
                      shared_page(p.accounts, seq, len, n, i);
  if (up < -1 || up >= i) up = -2;
  uint32_t set[kWords];
#pragma unroll
  for (int w = 0; w < kWords; ++w) set[w] = w == i >> 5 ? 1u << (i & 31) : 0u;
  // pointers lead to lower nodes only, so that they end within the tree's depth
  while (true) {
    above[i] = up;
#pragma unroll
    for (int w = 0; w < kWords; ++w) sets[w][i] = set[w];
    if (!__syncthreads_or(up >= 0)) break;
    if (up >= 0) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) set[w] |= sets[w][up];
      up = above[up];
    }
    __syncthreads();  // read before the next step writes
  }
  int depth = -1;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    if (up != -1) set[w] = 0u;
    depth += __popc(set[w]);
    sets[w][i] = set[w];
  }
  if (__syncthreads_or(shared)) {
    if (i == 0) flag_status(p.status, KV_NVFP4_DEV_SHARED_PAGE);
    no_place();
    return;
  }
  for (int x = i; x < n * W; x += 32 * kWords) p.mask[seq * n * W + x] = sets[x % W][x / W];
  if (p.slots != nullptr && i < n) {
    p.seq_ids[seq * n + i] = (int32_t)seq;
    p.slots[seq * n + i] = len + i;
    p.positions[seq * n + i] = first + (depth > 0 ? depth : 0);
  }
}

struct TreeAcceptParams {
  const int32_t* parents;   // [num_seqs][n]; null: path and count are given
  const int32_t* draft;     // [num_seqs][n]
  const int32_t* target;    // [num_seqs][n]
  const int32_t* expected;  // [num_seqs]
  const int32_t* lens;      // [num_seqs]
  const int32_t* block_table;
  int32_t n, max_pages, num_pages, Hkv;
  uint8_t* pool;            // null: nothing is moved
  int32_t* path;            // [num_seqs][n]
  int32_t* count;           // [num_seqs]
  int32_t* next;            // [num_seqs]
  int32_t* new_lens;        // [num_seqs], or null
  Accounts accounts;
  int32_t* status;
};

constexpr int kAcceptThreads = 256;
static_assert(kAcceptThreads >= kMaxNodes, "a thread per node");

// One CTA per sequence. One warp walks the tree, each lane holding eight nodes: the next node is the
// lowest one under the last whose drafted token is the awaited one (a warp minimum), and its target
// the token awaited next. Meanwhile the other threads fetch the page ids of the tree's slots. Then the
// path's rows move: eight threads per (row, KV head), 16 bytes of the K or V codes each, and the
// scales; in waves of ascending rows, each read whole before it is written. Row j comes from slot
// path[j] >= j of the tree and the path ascends, so a wave is written only over rows that no later
// wave reads.
//
// Bounds: the chain of dependent loads (lengths, tokens and page ids, then rows) and the launch. Replayed
// from a graph a tree of 16 takes 1.8 us, 64 trees of 64 with 4 KV heads 2.9, with 8 heads 3.4; called, the
// host's 6.4 to 6.6.
__global__ void __launch_bounds__(kAcceptThreads) tree_accept_kernel(const TreeAcceptParams p) {
  __shared__ int32_t path[kMaxNodes], target[kMaxNodes], pages[kTreePages];
  __shared__ int32_t walked[2];  // the path's length, the token behind it
  const int tid = threadIdx.x, lane = tid & 31, n = p.n;
  const int64_t seq = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int32_t base = p.lens[seq];
  const bool walk = p.parents != nullptr;
  int32_t count = walk ? 0 : p.count[seq];
  bool bad = base < 0 || (int64_t)base + n > (p.pool != nullptr ? (int64_t)p.max_pages * kPage : 0x7FFFFFFF);
  bad = bad || count < 0 || count > n;
  int32_t parent[kMaxNodes / 32], draft[kMaxNodes / 32], token = 0;
  if (walk) {
    if (tid < n) target[tid] = p.target[seq * n + tid];
    if (tid < 32) {
      token = p.expected[seq];
#pragma unroll
      for (int k = 0; k < kMaxNodes / 32; ++k) {
        const int i = lane + 32 * k;
        parent[k] = i < n ? p.parents[seq * n + i] : -2;
        if (parent[k] < -1 || parent[k] >= i) parent[k] = -2;
        draft[k] = i < n ? p.draft[seq * n + i] : 0;
      }
    }
  } else if (!bad) {  // the given path ascends within the tree
    int32_t node = 0;
    if (tid < count) {
      node = path[tid] = p.path[seq * n + tid];
      bad = node < 0 || node >= n || (tid > 0 && p.path[seq * n + tid - 1] >= node);
    }
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      flag_status(p.status, KV_NVFP4_DEV_BAD_POS);
      if (walk) p.count[seq] = 0;  // a further layer's call moves as many rows as it finds here
    }
    return;
  }
  const int first_page = base / kPage;
  bool shared = false;
  if (tid >= 32 && tid < 32 + kTreePages) {
    const int j = tid - 32;
    pages[j] = p.pool != nullptr && first_page + j < p.max_pages
                   ? p.block_table[seq * p.max_pages + first_page + j] : -1;
    shared = p.accounts.refs != nullptr && shared_page(p.accounts, seq, base, n, j);
  }
  const int32_t awaited = token;
  if (walk && tid < 32) {
    int at = -1, length = 0;
    while (true) {
      uint32_t best = 0xFFFFFFFFu;
#pragma unroll
      for (int k = kMaxNodes / 32 - 1; k >= 0; --k)
        if (parent[k] == at && draft[k] == token) best = (uint32_t)(lane + 32 * k);
      best = __reduce_min_sync(0xffffffffu, best);
      if (best == 0xFFFFFFFFu) break;  // nodes lie above their parents: at most n steps
      at = (int)best;
      if (lane == 0) path[length] = at;
      ++length;
      token = target[at];
    }
    if (lane == 0) {
      walked[0] = length;
      walked[1] = token;
    }
  }
  const bool none = __syncthreads_or(shared);  // in pages that others hold nothing is moved or accepted
  if (walk) count = walked[0];
  if (none) {
    count = 0;
    if (tid == 0) flag_status(p.status, KV_NVFP4_DEV_SHARED_PAGE);
  }
  if (walk) {
    if (tid < count) p.path[seq * n + tid] = path[tid];
    if (tid == 0) {
      p.count[seq] = count;
      p.next[seq] = none ? awaited : walked[1];
    }
  }
  if (tid == 0 && p.new_lens != nullptr) p.new_lens[seq] = base + count;
  if (p.pool == nullptr) return;
  // rows from the first one that is not in its place
  int stay = 0;
  stay = __syncthreads_count(tid < count && path[tid] == tid);
  const int64_t block = (int64_t)p.Hkv * 9216;
  const int q = tid & 7;  // K pieces 0 .. 3, V pieces 4 .. 7
  const int units = (count - stay) * p.Hkv;
  int32_t bad_page = 0;
  for (int u0 = 0; u0 < units; u0 += kAcceptThreads / 8) {
    const int u = u0 + (tid >> 3);
    const int j = stay + u / p.Hkv, head = u % p.Hkv;
    uint4 codes = make_uint4(0u, 0u, 0u, 0u);
    uint2 scales = make_uint2(0u, 0u);
    uint8_t* dst = nullptr;
    int to = 0;
    auto code_at = [&](int slot) {
      return q < 4 ? head * 4096 + (slot >> 3) * 512 + q * 128 + (slot & 7) * 16
                   : p.Hkv * 4608 + head * 4096 + slot * 64 + (q - 4) * 16;
    };
    auto v_scale_at = [&](int slot) { return p.Hkv * 8704 + head * 512 + slot * 8; };
    if (u < units) {
      const int from = base + path[j];
      to = base + j;
      const int32_t src_page = pages[from / kPage - first_page];
      const int32_t dst_page = pages[to / kPage - first_page];
      if (src_page < 0 || src_page >= p.num_pages || dst_page < 0 || dst_page >= p.num_pages) {
        bad_page = KV_NVFP4_DEV_BAD_PAGE;
      } else {
        const uint8_t* src = p.pool + src_page * block;
        dst = p.pool + dst_page * block;
        const int slot = from % kPage;
        codes = *reinterpret_cast<const uint4*>(src + code_at(slot));
        if (q < 2)
          scales.x = *reinterpret_cast<const uint32_t*>(src + kscale_offset(p.Hkv, head, slot, q));
        else if (q == 4)
          scales = *reinterpret_cast<const uint2*>(src + v_scale_at(slot));
      }
    }
    __syncthreads();  // the wave is read before it is written
    if (dst != nullptr) {
      const int slot = to % kPage;
      *reinterpret_cast<uint4*>(dst + code_at(slot)) = codes;
      if (q < 2)
        *reinterpret_cast<uint32_t*>(dst + kscale_offset(p.Hkv, head, slot, q)) = scales.x;
      else if (q == 4)
        *reinterpret_cast<uint2*>(dst + v_scale_at(slot)) = scales;
    }
  }
  if (bad_page != 0) flag_status(p.status, bad_page);
}

Accounts accounts_of(const kv_nvfp4_pages* p) {
  if (p == nullptr) return Accounts{nullptr, nullptr, 0, 0};
  return Accounts{p->block_table, p->refs, p->max_pages, p->num_pages};
}

cudaLaunchAttribute programmatic() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

}  // namespace

cudaError_t launch_tree_mask(const int32_t* parents, int32_t num_seqs, int32_t n,
                             const int32_t* lens, const int32_t* first_pos, uint32_t* mask,
                             int32_t* seq_ids, int32_t* slots, int32_t* positions,
                             const kv_nvfp4_pages* pages, int32_t* status, cudaStream_t stream) {
  const TreeMaskParams p{parents,   lens, first_pos, mask, seq_ids, slots,
                         positions, accounts_of(pages), n, status};
  cudaLaunchAttribute attr[1] = {programmatic()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_seqs);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int words = n <= 32 ? 1 : n <= 64 ? 2 : n <= 128 ? 4 : kMaxWords;
  cfg.blockDim = dim3(32u * words);
  switch (words) {
    case 1: return cudaLaunchKernelEx(&cfg, tree_mask_kernel<1>, p);
    case 2: return cudaLaunchKernelEx(&cfg, tree_mask_kernel<2>, p);
    case 4: return cudaLaunchKernelEx(&cfg, tree_mask_kernel<4>, p);
    default: return cudaLaunchKernelEx(&cfg, tree_mask_kernel<kMaxWords>, p);
  }
}

cudaError_t launch_tree_accept(const int32_t* parents, const int32_t* draft, const int32_t* target,
                               const int32_t* expected, int32_t num_seqs, int32_t n,
                               const int32_t* lens, const int32_t* block_table, int32_t max_pages,
                               int32_t num_pages, uint8_t* pool, int32_t* path, int32_t* count,
                               int32_t* next, int32_t* new_lens, const kv_nvfp4_pages* pages,
                               int32_t Hkv, int32_t* status, cudaStream_t stream) {
  const TreeAcceptParams p{parents, draft, target, expected, lens, block_table, n, max_pages, num_pages,
                           Hkv, pool, path, count, next, new_lens, accounts_of(pages), status};
  cudaLaunchAttribute attr[1] = {programmatic()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_seqs);
  cfg.blockDim = dim3(kAcceptThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_accept_kernel, p);
}

}  // namespace kvnvfp4
