// Page accounts of sequences that share a pool: which pages each one holds, how many hold each page,
// and the stack of free pages (kv_nvfp4_pages_init, _fork, _resize), and the copy of pages that a
// resize asks for (kv_nvfp4_copy_pages). No counterpart in the pages.
//
// Everything is decided in one order, sequence by sequence and place by place, so that equal calls
// give equal tables: counts go up and down by integer atomics, whose order does not show, and what is
// taken from the stack or pushed onto it is ranked by prefix sums.
//
// Each kernel lets the launch of the next one on the stream begin while it runs; that one waits for its
// end before it reads anything (two resizes for 4 sessions, back to back in a graph: 8.1 -> 7.0 us).

#include <cstdint>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"

namespace kvnvfp4 {

namespace {

// The workspace: per page, the call (high word) and the place in its order (low word) of the last
// drop; per page, the last call that found it shared; per page, a page freed by the call; the calls
// so far that left such marks. A mark counts if its call is the present one. Numbers are 1 to 2^32 - 1:
// the call behind the last one clears the marks and is number 1 again.
struct PagesWork {
  unsigned long long* last_drop;
  uint32_t* shared_in;
  int32_t* freed;
  uint32_t* calls;
};

__host__ __device__ inline PagesWork pages_work(void* workspace, int64_t num_pages) {
  PagesWork w;
  w.last_drop = static_cast<unsigned long long*>(workspace);
  w.shared_in = reinterpret_cast<uint32_t*>(w.last_drop + num_pages);
  w.freed = reinterpret_cast<int32_t*>(w.shared_in + num_pages);
  w.calls = reinterpret_cast<uint32_t*>(w.freed + num_pages);
  return w;
}

__global__ void __launch_bounds__(256) pages_init_kernel(const kv_nvfp4_pages p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  const PagesWork w = pages_work(p.workspace, p.num_pages);
  for (int64_t i = first; i < p.num_pages; i += step) {
    p.refs[i] = 0;
    p.free_list[i] = (int32_t)(p.num_pages - 1 - i);  // page 0 is taken first
    w.last_drop[i] = 0;
    w.shared_in[i] = 0;
  }
  for (int64_t i = first; i < (int64_t)p.num_seqs * p.max_pages; i += step) p.block_table[i] = -1;
  for (int64_t i = first; i < p.num_seqs; i += step) p.held[i] = 0;
  if (first == 0) {
    *p.free_count = p.num_pages;
    *w.calls = 0;
  }
}

struct ForkParams {
  kv_nvfp4_pages p;
  const int32_t* src;   // [n]
  const int32_t* dst;   // [n]
  const int32_t* lens;  // [n]
  int32_t n;
  int32_t* status;
};

constexpr int kForkThreads = 512;

// One CTA per fork: the row's entries copied, the pages' counts raised. A fork reads only what no other
// fork of the call writes: its own target's count of pages, and its source's row, which must not be any
// fork's target (of two that name the same target only the first is carried out). Bounds: the loads one
// behind the other and the counts' atomics (8 forks of 1563 pages 2.4 us back to back, 4.8 alone).
__global__ void __launch_bounds__(kForkThreads) pages_fork_kernel(const ForkParams f) {
  const kv_nvfp4_pages& p = f.p;
  const int tid = threadIdx.x, i = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int32_t src = f.src[i], dst = f.dst[i], len = f.lens[i];
  bool bad = src < 0 || src >= p.num_seqs || dst < 0 || dst >= p.num_seqs;
  for (int j = tid; j < f.n; j += kForkThreads) {
    const int32_t other = f.dst[j];
    bad = bad || other == src || (j < i && other == dst);
  }
  const bool inside = src >= 0 && src < p.num_seqs && dst >= 0 && dst < p.num_seqs;
  const int32_t have = inside ? p.held[dst] : 0, room = inside ? p.held[src] : 0;
  // (the barrier also stands between the reads of held[dst] and its write)
  if (__syncthreads_or(bad || have != 0)) {
    if (tid == 0) flag_status(f.status, KV_NVFP4_DEV_BAD_SEQ);
    return;
  }
  const int32_t pages = len < 0 ? -1 : (int32_t)(((int64_t)len + kPage - 1) / kPage);
  if (pages < 0 || pages > room || pages > p.max_pages) {
    if (tid == 0) flag_status(f.status, KV_NVFP4_DEV_BAD_POS);
    return;
  }
  const int32_t* from = p.block_table + (int64_t)src * p.max_pages;
  int32_t* to = p.block_table + (int64_t)dst * p.max_pages;
  bool lost = false;
  for (int j = tid; j < pages; j += kForkThreads) {
    const int32_t page = from[j];
    to[j] = page;
    if (page >= 0 && page < p.num_pages) atomicAdd(p.refs + page, 1);
    else lost = true;
  }
  if (lost) flag_status(f.status, KV_NVFP4_DEV_BAD_PAGE);
  if (tid == 0) p.held[dst] = pages;
}

struct ResizeParams {
  kv_nvfp4_pages p;
  const int32_t* keep;   // [num_seqs]
  const int32_t* room;   // [num_seqs]
  int32_t* copies;       // [num_seqs][2]
  int32_t* kept;         // [num_seqs] keep, or -1 for a refused sequence; or null
  int32_t* status;
};

constexpr int kResizeThreads = 1024;
constexpr int kResizeMaxCluster = 8;

// Every thread of the cluster meets; what was written before is read after it.
__device__ __forceinline__ void cluster_meet() {
  __syncthreads();
  cluster_arrive();
  cluster_wait();
}
// A word of this CTA's shared memory as the cluster's CTA `rank` has it.
__device__ __forceinline__ uint32_t peer_word(const void* shared, uint32_t rank) {
  return cluster_load(cluster_peer(smem_u32(shared), rank));
}

// Exclusive sum over the block's threads, and the block's sum; v < 2^31 in all.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the sums of a scan before have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  const uint32_t mine = warp_sums[lane];  // 32 warps
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0u);
  total = __reduce_add_sync(0xffffffffu, mine);
  return before + x - v;
}

// The number of the block's threads before this one with v set, and of all of them.
__device__ __forceinline__ uint32_t block_rank(bool v, uint32_t* warp_sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t set = __ballot_sync(0xffffffffu, v);
  __syncthreads();  // the sums of a scan before have been read
  if (lane == 0) warp_sums[warp] = __popc(set);
  __syncthreads();
  const uint32_t mine = warp_sums[lane];  // 32 warps
  total = __reduce_add_sync(0xffffffffu, mine);
  return __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0u) + __popc(set & ((1u << lane) - 1u));
}

// A resize of at most one entry per thread, by one CTA: everything stays in registers. The cluster meets
// once, before the first write, so that no CTA reads the sequences' numbers behind it. A page that
// several rows drop is freed by whoever lowers its count to zero, in the place of its last drop, which
// that thread looks up. Bounds: about ten dependent loads and barriers, 3.9 us (4 sessions) to 4.6 (256)
// of a resize back to back; in the cluster's form below 10 to 12.
struct FewEntries {
  int32_t top[kResizeThreads];         // the stack from its top on
  int32_t dropped[kResizeThreads];     // page dropped by each entry, or -1
  uint32_t takes_before[kResizeThreads + 1];
  uint8_t freed[kResizeThreads];
  uint32_t warp_sums[32];
  uint32_t all_taken;
};

template <class SeqOf, class PlaceOf>
__device__ __forceinline__ void resize_few(const ResizeParams& r, FewEntries& sh,
                                           const int32_t* before, const int32_t* need_of,
                                           const int32_t* held_of, SeqOf seq_of, PlaceOf place_of,
                                           uint32_t entries, int32_t free_now, int32_t bad) {
  const kv_nvfp4_pages& p = r.p;
  const int tid = threadIdx.x, S = p.num_seqs;
  const uint32_t e = (uint32_t)tid;
  const int32_t top = tid < free_now ? p.free_list[free_now - 1 - tid] : -1;
  sh.freed[tid] = 0;
  if (tid == 0) sh.all_taken = 0;
  int s = 0, j = 0;
  int32_t page = -1, refs = 0, keep = 0;
  bool take = false, drop = false, in_pool = false;
  if (e < entries) {
    s = seq_of(e);
    j = place_of(s, e);
    keep = r.keep[s];
    if (j < held_of[s]) {
      page = p.block_table[(int64_t)s * p.max_pages + j];
      in_pool = page >= 0 && page < p.num_pages;
      if (in_pool) refs = p.refs[page];
      else bad |= KV_NVFP4_DEV_BAD_PAGE;
      drop = j >= need_of[s] || (in_pool && refs > 1);
      take = drop && j < need_of[s];
    } else {
      take = true;
    }
  }
  uint32_t wanted;
  const uint32_t at = block_rank(take, sh.warp_sums, wanted);
  sh.takes_before[tid] = at;
  sh.top[tid] = top;
  if (tid == 0) sh.takes_before[entries] = wanted;
  __syncthreads();
  // a sequence's demand with those before it
  auto met = [&](int seq, uint32_t& upto) {
    upto = sh.takes_before[before[seq + 1]];
    return upto == sh.takes_before[before[seq]] || upto <= (uint32_t)free_now;
  };
  uint32_t upto = 0;
  if (e < entries) {
    const bool ok = met(s, upto);
    if (ok && take) atomicMax(&sh.all_taken, upto);
    if (!ok) {
      bad |= KV_NVFP4_DEV_NO_PAGE;
      if (r.kept != nullptr) r.kept[s] = -1;  // (one that is not met has entries)
    }
    take = take && ok;
    drop = drop && ok;
  }
  cluster_wait();  // every CTA has read the sequences' numbers and has seen that there is one for one CTA
  const bool lowers = drop && in_pool;
  const int32_t was = lowers ? atomicSub(p.refs + page, 1) : 0;  // behind every read of the counts
  sh.dropped[tid] = lowers ? page : -1;
  __syncthreads();
  if (lowers && was == 1) {
    uint32_t last = e;
    if (refs > 1)
      for (last = entries - 1; sh.dropped[last] != page; --last) {}
    sh.freed[last] = 1;
  }
  __syncthreads();
  const bool freed = sh.freed[tid] != 0;
  uint32_t all_freed;
  const uint32_t rank = block_rank(freed, sh.warp_sums, all_freed);
  const uint32_t left = (uint32_t)free_now - sh.all_taken;
  if (freed && left + rank < (uint32_t)p.num_pages) p.free_list[left + rank] = page;
  if (take || drop) {
    int32_t fresh = -1;
    if (take) {
      fresh = sh.top[at];
      if (fresh >= 0 && fresh < p.num_pages) p.refs[fresh] = 1;
      else bad |= KV_NVFP4_DEV_BAD_PAGE;
      if (drop && (int64_t)j * kPage < keep) {
        r.copies[2 * s] = page;
        r.copies[2 * s + 1] = fresh;
      }
    }
    p.block_table[(int64_t)s * p.max_pages + j] = fresh;
  }
  for (int q = tid; q < S; q += kResizeThreads)
    if (held_of[q] != need_of[q] && met(q, upto)) p.held[q] = need_of[q];
  if (tid == 0) *p.free_count = (int32_t)min(left + all_freed, (uint32_t)p.num_pages);
  if (bad != 0) flag_status(r.status, bad);
}

// A resize of at most kShareEntries entries per thread of the cluster whose demand the stack meets
// (else false, with nothing changed): each entry is looked at once and stays in registers. The cluster
// meets when the counts have been read, when the last drops of pages with several holders are noted
// (only if there are any), when the freed entries are counted, and before it ends. Bounds: these meetings
// and the loads between them, 9 us for 8192 entries of 4 sessions (12 with every entry looked at in
// each step, as in the general form below; in a cluster of 4 the same, one CTA by the general form 35).
constexpr int kShareEntries = 4;

template <class SeqOf, class PlaceOf>
__device__ __forceinline__ bool resize_shares(const ResizeParams& r, const PagesWork& w, uint32_t call,
                                              uint32_t* warp_sums, uint32_t* out_counts,
                                              const int32_t* before, const int32_t* need_of,
                                              const int32_t* held_of, SeqOf seq_of, PlaceOf place_of,
                                              uint32_t entries, int32_t free_now, int32_t bad) {
  const kv_nvfp4_pages& p = r.p;
  const int tid = threadIdx.x, S = p.num_seqs;
  const uint32_t C = cluster_size(), rank = cluster_rank();
  const uint32_t share = max((entries + C - 1) / C, (uint32_t)kResizeThreads);
  const uint32_t e_lo = min(entries, rank * share), e_hi = min(entries, e_lo + share);
  int32_t seq[kShareEntries], place[kShareEntries], page[kShareEntries], other[kShareEntries];
  uint32_t at[kShareEntries];
  bool take[kShareEntries], drop[kShareEntries];  // drop: of a page in the pool
  bool gone[kShareEntries];                       // the place is emptied
#pragma unroll
  for (int u = 0; u < kShareEntries; ++u) {
    const uint32_t e = e_lo + u * kResizeThreads + tid;
    seq[u] = place[u] = 0;
    page[u] = -1;
    take[u] = drop[u] = gone[u] = false;
    if (e >= e_hi) continue;
    seq[u] = seq_of(e);
    place[u] = place_of(seq[u], e);
    take[u] = place[u] >= held_of[seq[u]];
    gone[u] = !take[u] && place[u] >= need_of[seq[u]];
    if (!take[u]) page[u] = p.block_table[(int64_t)seq[u] * p.max_pages + place[u]];
  }
  bool some = false;
#pragma unroll
  for (int u = 0; u < kShareEntries; ++u) {
    const bool in_pool = page[u] >= 0 && page[u] < p.num_pages;
    const bool real = e_lo + u * kResizeThreads + tid < e_hi;
    other[u] = in_pool ? __ldcg(p.refs + page[u]) : 1;
    if (real && !take[u] && !in_pool) bad |= KV_NVFP4_DEV_BAD_PAGE;
    drop[u] = in_pool && (gone[u] || other[u] > 1);
    if (drop[u] && !gone[u]) take[u] = true;
    some = some || (drop[u] && other[u] > 1);
  }
  uint32_t taken = 0, sum;
#pragma unroll
  for (int u = 0; u < kShareEntries; ++u) {
    at[u] = 0;
    if (e_lo + u * kResizeThreads >= e_hi) continue;  // for the whole CTA
    at[u] = taken + block_rank(take[u], warp_sums, sum);
    taken += sum;
  }
  some = __syncthreads_or(some);
  if (tid == 0) {
    out_counts[1] = taken;
    out_counts[2] = some;
  }
  cluster_meet();  // the counts of holders have been read
  uint32_t taken_before = 0, all_taken = 0;
  bool shared = false;
  for (uint32_t c = 0; c < C; ++c) {
    const uint32_t n = peer_word(&out_counts[1], c);
    if (c < rank) taken_before += n;
    all_taken += n;
    shared = shared || peer_word(&out_counts[2], c) != 0u;
  }
  if (all_taken > (uint32_t)free_now) return false;  // the same for the whole cluster

  int32_t fresh[kShareEntries];
#pragma unroll
  for (int u = 0; u < kShareEntries; ++u) {
    const uint32_t e = e_lo + u * kResizeThreads + tid;
    fresh[u] = take[u] ? p.free_list[free_now - 1 - (int32_t)(taken_before + at[u])] : -1;
    if (drop[u]) {
      atomicSub(p.refs + page[u], 1);
      if (other[u] > 1) atomicMax(w.last_drop + page[u], ((unsigned long long)call << 32) | (e + 1));
    }
  }
  if (shared) cluster_meet();  // the counts are lowered, the last drops noted
  uint32_t freed = 0;
#pragma unroll
  for (int u = 0; u < kShareEntries; ++u) {
    const uint32_t e = e_lo + u * kResizeThreads + tid;
    if (drop[u] && other[u] > 1)  // the last holder's, in the place of the last drop
      drop[u] = __ldcg(p.refs + page[u]) == 0 &&
                __ldcg(w.last_drop + page[u]) == (((unsigned long long)call << 32) | (e + 1));
    if (e_lo + u * kResizeThreads >= e_hi) continue;
    at[u] = freed + block_rank(drop[u], warp_sums, sum);
    freed += sum;
  }
  if (tid == 0) out_counts[0] = freed;
  cluster_meet();  // the stack's top has been read
  uint32_t freed_before = 0, all_freed = 0;
  for (uint32_t c = 0; c < C; ++c) {
    const uint32_t n = peer_word(&out_counts[0], c);
    if (c < rank) freed_before += n;
    all_freed += n;
  }
  cluster_arrive();  // awaited at the end
  const uint32_t left = (uint32_t)free_now - all_taken;
#pragma unroll
  for (int u = 0; u < kShareEntries; ++u) {
    const uint32_t to = left + freed_before + at[u];
    if (drop[u] && to < (uint32_t)p.num_pages) p.free_list[to] = page[u];
    if (!take[u] && !gone[u]) continue;
    if (take[u]) {
      if (fresh[u] >= 0 && fresh[u] < p.num_pages) p.refs[fresh[u]] = 1;
      else bad |= KV_NVFP4_DEV_BAD_PAGE;
      if (page[u] >= 0 && (int64_t)place[u] * kPage < r.keep[seq[u]]) {
        r.copies[2 * seq[u]] = page[u];
        r.copies[2 * seq[u] + 1] = fresh[u];
      }
    }
    p.block_table[(int64_t)seq[u] * p.max_pages + place[u]] = fresh[u];
  }
  for (int q = (int)(rank * kResizeThreads) + tid; q < S; q += (int)(C * kResizeThreads))
    if (held_of[q] != need_of[q]) p.held[q] = need_of[q];
  if (rank == 0 && tid == 0) {
    *p.free_count = (int32_t)min(left + all_freed, (uint32_t)p.num_pages);
    *w.calls = call;
  }
  if (bad != 0) flag_status(r.status, bad);
  cluster_wait();
  return true;
}

// One cluster. The entries that a call can touch (places keep / 64 .. max(held, need) of every sequence)
// lie end to end in the order of sequences and places; a CTA takes a contiguous share of them, and
// every CTA knows every sequence's numbers (it works them out itself). An entry is
//   dropped  behind the new need, or shared (more than one holder before the call) although it is to be
//            written,
//   taken    behind what the sequence held, or in the place of a shared one.
// Steps, with a meeting of the cluster after each: shared entries found and the sequences' demands
// summed up, so that it is known who gets pages; counts lowered, each page's last drop noted; freed
// (dropped last, nobody left) and taken entries counted; the freed pages listed and the fresh ones
// entered by rank; the list pushed onto the stack.
//
// Two shorter forms above: at most 1024 entries, and at most 4096 per CTA that the stack can serve. What is
// left, tens of thousands of entries or a stack that runs out, is bound by the search for an entry's
// sequence, its page and its count in four passes, the first of them over all entries in every CTA: 31
// of 32 sessions on one prompt of 100000 tokens end (48453 shared entries) in 46 us, 63 of 64 (98469) in
// 93; 8 of 9 (12504, the form above) in 11.
__global__ void __launch_bounds__(kResizeThreads) pages_resize_kernel(const ResizeParams r) {
  extern __shared__ int32_t per_seq[];  // [num_seqs + 1] entries before, [num_seqs] need, held, demand
  __shared__ uint32_t warp_sums[32];
  __shared__ uint32_t out_counts[3];    // freed and taken entries of this CTA's share, and whether one
                                        // is dropped from among several holders
  __shared__ uint32_t all_taken;
  __shared__ FewEntries few;
  const kv_nvfp4_pages& p = r.p;
  const int tid = threadIdx.x, S = p.num_seqs;
  const uint32_t C = cluster_size(), rank = cluster_rank();
  int32_t* const before = per_seq;
  int32_t* const need_of = before + S + 1;
  int32_t* const held_of = need_of + S;
  int32_t* const demand = held_of + S;  // then 1: gets its pages, 0: stays as it was
  const PagesWork w = pages_work(p.workspace, p.num_pages);
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint32_t call = __ldcg(w.calls) + 1;
  const int32_t stack = __ldcg(p.free_count);
  const int32_t free_now = stack < 0 ? 0 : stack > p.num_pages ? p.num_pages : stack;
  if (tid == 0) all_taken = 0;
  int32_t bad = stack != free_now ? KV_NVFP4_DEV_BAD_PAGE : 0;

  // the sequences' numbers; one that is refused has no entries
  uint32_t entries = 0;
  for (int s0 = 0; s0 < S; s0 += kResizeThreads) {
    const int s = s0 + tid;
    uint32_t n = 0;
    if (s < S) {
      const int32_t keep = r.keep[s], room = r.room[s], held = p.held[s];
      const int32_t need = (int32_t)(((int64_t)room + kPage - 1) / kPage);
      const bool ok = keep >= 0 && room >= keep && need <= p.max_pages && held >= 0 &&
                      held <= p.max_pages && ((int64_t)keep + kPage - 1) / kPage <= held;
      if (!ok) bad |= KV_NVFP4_DEV_BAD_POS;
      const int32_t full = ok ? keep / kPage : 0;
      n = ok ? (uint32_t)(max(held, need) - full) : 0u;
      need_of[s] = ok ? need : 0;
      held_of[s] = ok ? held : 0;
      demand[s] = ok ? max(0, need - held) : 0;
      if (rank == 0) {
        r.copies[2 * s] = r.copies[2 * s + 1] = -1;
        if (r.kept != nullptr) r.kept[s] = ok ? keep : -1;  // (who gets pages is found out below)
      }
    }
    uint32_t sum;
    const uint32_t at = block_scan(n, warp_sums, sum);
    if (s < S) before[s] = (int32_t)(entries + at);
    entries += sum;
  }
  if (tid == 0) before[S] = (int32_t)entries;
  __syncthreads();
  // the sequence and place of entry e
  auto seq_of = [&](uint32_t e) {
    int lo = 0, hi = S;  // before[lo] <= e < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((uint32_t)before[mid] <= e) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  auto place_of = [&](int s, uint32_t e) {
    const int last = max(held_of[s], need_of[s]);
    return last - (before[s + 1] - (int32_t)e);
  };
  auto inside = [&](int32_t page) { return page >= 0 && page < p.num_pages; };

  if (entries <= (uint32_t)kResizeThreads) {  // the same for every CTA
    // (nothing written is read behind this meeting, and what was read has been branched on: no release,
    // which takes 0.3 us)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    if (rank == 0) resize_few(r, few, before, need_of, held_of, seq_of, place_of, entries, free_now, bad);
    else cluster_wait();
    return;
  }

  if (call == 0) {  // the same for every CTA
    for (int64_t i = rank * kResizeThreads + tid; i < p.num_pages; i += C * kResizeThreads) {
      w.last_drop[i] = 0;
      w.shared_in[i] = 0;
    }
    cluster_meet();
    call = 1;
  }

  if (entries <= C * (uint32_t)(kResizeThreads * kShareEntries) &&
      resize_shares(r, w, call, warp_sums, out_counts, before, need_of, held_of, seq_of, place_of,
                    entries, free_now, bad))
    return;

  // shared entries, found by every CTA for itself (mostly one per sequence is looked at)
  for (uint32_t e = tid; e < entries; e += kResizeThreads) {
    const int s = seq_of(e), j = place_of(s, e);
    if (j >= min(held_of[s], need_of[s])) continue;
    const int32_t page = p.block_table[(int64_t)s * p.max_pages + j];
    if (!inside(page)) {
      bad |= KV_NVFP4_DEV_BAD_PAGE;
    } else if (__ldcg(p.refs + page) > 1) {
      w.shared_in[page] = call;
      atomicAdd(&demand[s], 1);
    }
  }
  __syncthreads();
  // who gets pages: the sequences up to the first whose demand, with those before it, is not met
  uint32_t wanted = 0;
  for (int s0 = 0; s0 < S; s0 += kResizeThreads) {
    const int s = s0 + tid;
    const uint32_t d = s < S ? (uint32_t)demand[s] : 0u;
    uint32_t sum;
    const uint32_t upto = wanted + block_scan(d, warp_sums, sum) + d;
    const bool ok = d == 0 || upto <= (uint32_t)free_now;
    if (s < S) {
      if (!ok) {
        bad |= KV_NVFP4_DEV_NO_PAGE;
        if (rank == 0 && r.kept != nullptr) r.kept[s] = -1;
      }
      if (ok && d > 0) atomicMax(&all_taken, upto);
      demand[s] = ok;
    }
    wanted += sum;
  }
  cluster_meet();

  // this CTA's share
  uint32_t share = (entries + C - 1) / C;
  share = max(share, (uint32_t)kResizeThreads);
  const uint32_t e_lo = min(entries, rank * share), e_hi = min(entries, e_lo + share);
  struct Entry {
    int s, j;
    int32_t page;
    bool drop, take;
  };
  auto entry = [&](uint32_t e) {
    Entry x;
    x.s = seq_of(e);
    x.j = place_of(x.s, e);
    const int held = held_of[x.s], need = need_of[x.s];
    x.page = -1;
    x.drop = x.take = false;
    if (demand[x.s] == 0) return x;
    if (x.j >= held) {
      x.take = true;
    } else {
      x.page = p.block_table[(int64_t)x.s * p.max_pages + x.j];
      if (x.j >= need) x.drop = true;
      else if (inside(x.page) && __ldcg(w.shared_in + x.page) == call) x.drop = x.take = true;
    }
    return x;
  };
  auto mark_of = [&](uint32_t e) { return ((unsigned long long)call << 32) | (e + 1); };
  for (uint32_t e = e_lo + tid; e < e_hi; e += kResizeThreads) {
    const Entry x = entry(e);
    if (!x.drop) continue;
    if (inside(x.page)) {
      atomicSub(p.refs + x.page, 1);
      atomicMax(w.last_drop + x.page, mark_of(e));
    } else {
      bad |= KV_NVFP4_DEV_BAD_PAGE;
    }
  }
  cluster_meet();

  auto freed_by = [&](const Entry& x, uint32_t e) {
    return x.drop && inside(x.page) && __ldcg(w.last_drop + x.page) == mark_of(e) &&
           __ldcg(p.refs + x.page) == 0;
  };
  uint32_t n_freed = 0, n_taken = 0;
  for (uint32_t e0 = e_lo; e0 < e_hi; e0 += kResizeThreads) {
    const uint32_t e = e0 + tid;
    bool freed = false, taken = false;
    if (e < e_hi) {
      const Entry x = entry(e);
      freed = freed_by(x, e);
      taken = x.take;
    }
    n_freed += __syncthreads_count(freed);
    n_taken += __syncthreads_count(taken);
  }
  if (tid == 0) {
    out_counts[0] = n_freed;
    out_counts[1] = n_taken;
  }
  cluster_meet();
  uint32_t freed_before = 0, taken_before = 0, all_freed = 0;
  for (uint32_t c = 0; c < C; ++c) {
    const uint32_t a = peer_word(&out_counts[0], c), b = peer_word(&out_counts[1], c);
    if (c < rank) {
      freed_before += a;
      taken_before += b;
    }
    all_freed += a;
  }
  for (uint32_t e0 = e_lo; e0 < e_hi; e0 += kResizeThreads) {
    const uint32_t e = e0 + tid;
    Entry x;
    x.drop = x.take = false;
    bool freed = false;
    if (e < e_hi) {
      x = entry(e);
      freed = freed_by(x, e);
    }
    uint32_t sum;
    const uint32_t at = block_scan((freed ? 1u << 16 : 0u) + (x.take ? 1u : 0u), warp_sums, sum);
    if (freed) w.freed[freed_before + (at >> 16)] = x.page;
    if (x.drop || x.take) {
      int32_t fresh = -1;
      if (x.take) {
        fresh = p.free_list[free_now - 1 - (int32_t)(taken_before + (at & 0xFFFFu))];
        if (inside(fresh)) p.refs[fresh] = 1;
        else bad |= KV_NVFP4_DEV_BAD_PAGE;
        if (x.drop && (int64_t)x.j * kPage < r.keep[x.s]) {
          r.copies[2 * x.s] = x.page;
          r.copies[2 * x.s + 1] = fresh;
        }
      }
      p.block_table[(int64_t)x.s * p.max_pages + x.j] = fresh;
    }
    freed_before += sum >> 16;
    taken_before += sum & 0xFFFFu;
  }
  cluster_meet();  // the stack's top has been read, the freed pages are listed

  const uint32_t left = (uint32_t)free_now - all_taken;
  for (uint32_t i = rank * kResizeThreads + tid; i < all_freed; i += C * kResizeThreads)
    if (left + i < (uint32_t)p.num_pages) p.free_list[left + i] = __ldcg(w.freed + i);
  for (int s = (int)(rank * kResizeThreads) + tid; s < S; s += (int)(C * kResizeThreads))
    if (demand[s] != 0 && (held_of[s] != need_of[s])) p.held[s] = need_of[s];
  if (rank == 0 && tid == 0) {
    *p.free_count = (int32_t)min(left + all_freed, (uint32_t)p.num_pages);
    *w.calls = call;
  }
  if (bad != 0) flag_status(r.status, bad);
}

// One CTA per (pair, KV head's share of the page): every load before the stores. Bounds: the launch and
// one round of loads (8 pages of 4 heads 3.5 us).
constexpr int kPairThreads = 192;
constexpr int kPairWords = 9216 / 16 / kPairThreads;

__global__ void __launch_bounds__(kPairThreads) copy_pages_kernel(uint8_t* pool,
                                                                  const int32_t* pairs, int32_t n,
                                                                  int32_t num_pages, int32_t Hkv,
                                                                  int32_t* status) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int64_t unit = blockIdx.x; unit < (int64_t)n * Hkv; unit += gridDim.x) {
    const int64_t i = unit / Hkv, part = unit % Hkv;
    const int32_t src = pairs[2 * i], dst = pairs[2 * i + 1];
    if (src == -1 && dst == -1) continue;
    if (src < 0 || src >= num_pages || dst < 0 || dst >= num_pages) {
      if (threadIdx.x == 0 && part == 0) flag_status(status, KV_NVFP4_DEV_BAD_PAGE);
      continue;
    }
    const uint4* from =
        reinterpret_cast<const uint4*>(pool + ((int64_t)src * Hkv + part) * 9216) + threadIdx.x;
    uint4* to = reinterpret_cast<uint4*>(pool + ((int64_t)dst * Hkv + part) * 9216) + threadIdx.x;
    uint4 v[kPairWords];
#pragma unroll
    for (int k = 0; k < kPairWords; ++k) v[k] = from[k * kPairThreads];
#pragma unroll
    for (int k = 0; k < kPairWords; ++k) to[k * kPairThreads] = v[k];
  }
}

cudaError_t launch(const void* kernel, int grid, int threads, size_t shared, int cluster,
                   void** args, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

}  // namespace

uint64_t pages_workspace_bytes(int32_t num_pages) { return 16ull * (uint64_t)num_pages + 16; }

cudaError_t launch_pages_init(const kv_nvfp4_pages* p, int32_t num_sms, cudaStream_t stream) {
  const int64_t most = (int64_t)p->num_seqs * p->max_pages > p->num_pages
                           ? (int64_t)p->num_seqs * p->max_pages : p->num_pages;
  const int64_t grid = (most + 255) / 256, full = 8ll * num_sms;
  void* args[] = {const_cast<kv_nvfp4_pages*>(p)};
  return launch((const void*)pages_init_kernel, (int)(grid < full ? grid : full), 256, 0, 0, args,
                stream);
}

cudaError_t launch_pages_fork(const kv_nvfp4_pages* p, const int32_t* src, const int32_t* dst,
                              const int32_t* lens, int32_t n, int32_t* status,
                              cudaStream_t stream) {
  ForkParams f{*p, src, dst, lens, n, status};
  void* args[] = {&f};
  return launch((const void*)pages_fork_kernel, n, kForkThreads, 0, 0, args, stream);
}

cudaError_t launch_pages_resize(const kv_nvfp4_pages* p, const int32_t* keep, const int32_t* room,
                                int32_t* copies, int32_t* kept, int32_t* status,
                                cudaStream_t stream) {
  static bool attr_done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  if (dev < 0 || dev >= 64 || !attr_done[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(pages_resize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (4 * KV_NVFP4_MAX_ACCOUNTED_SEQS + 1) * 4);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev] = true;
  }
  ResizeParams r{*p, keep, room, copies, kept, status};
  void* args[] = {&r};
  // the lengths are on the device: sized for the most entries that the table has
  int C = 1;
  while (C < kResizeMaxCluster && (int64_t)C * kResizeThreads < (int64_t)p->num_seqs * p->max_pages)
    C *= 2;
  return launch((const void*)pages_resize_kernel, C, kResizeThreads,
                (size_t)(4 * p->num_seqs + 1) * 4, C, args, stream);
}

cudaError_t launch_copy_pages(uint8_t* pool, const int32_t* pairs, int32_t n, int32_t num_pages,
                              int32_t Hkv, int32_t num_sms, int32_t* status, cudaStream_t stream) {
  void* args[] = {&pool, &pairs, &n, &num_pages, &Hkv, &status};
  const int64_t units = (int64_t)n * Hkv, full = 8ll * num_sms;
  return launch((const void*)copy_pages_kernel, (int)(units < full ? units : full), kPairThreads, 0,
                0, args, stream);
}

}  // namespace kvnvfp4
