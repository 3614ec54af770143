// Per-key weights from stored scores, for kv_nvfp4_decode_attn_weights when a KV head has at most 8
// query rows: in the launch after either form of the decode kernel (with groups over all KV heads, or
// of one). The attention kernel leaves the raw scores of every page it visits (-inf where a row does
// not see the key), [page][R rows][64 keys] per KV head; here one thread takes four keys and adds, row
// by row,
//   exp2((s - m_r) c2) / l_r
// onto the accounts. The row statistics come from the split-K partials themselves, so this work
// needs no merge before it: it runs in the same launch as the merge of the outputs.
//
// For 6 rows the scores are 24 bytes per key and KV head, written once and read once, against 72
// bytes of K to read again and a second Q.K^T (the call of 4 x 131072 tokens: 75.7 us, and 124 us
// with the weight pass in its first form); most of them stay in the L2 between the kernels (the pages
// of the cache are marked first for eviction). The scores' stores cost the attention kernel nothing
// that could be measured; what is left beside it, about 13 us, is a launch, the statistics and the
// way of 50 MB of scores through the L2. It is not the loads' latency: bulk copies of the scores into
// a ring in shared memory, two to four times as many bytes in flight, took the same 75.7 us.
#pragma once

#include "nvfp4_device.cuh"

namespace kvnvfp4 {

constexpr int kAccThreads = 256;
constexpr int kAccPages = kAccThreads / 16;  // pages of a CTA: 16 threads per page, 4 keys each
constexpr int kAccRows = 8;
// Four (64 registers: 56 bytes of spills, 88 in the tile plan's kernel) took a decode call of 4 x
// 131072 tokens 78.0 us, three (80 registers: none, and 8 bytes) 73.5, two 74.5; twice as many, shorter
// CTAs 76.3 (in one run; 75.7 for three since)
constexpr int kAccCtasPerSm = 3;

struct AccountParams {
  const float* scores;     // [pages of all groups][heads per group][R][64]
  const float2* stats;     // [num_seqs][Hkv][R]: (m, 1 / l) of rows of unsplit groups
  const float* w_in;       // [num_seqs][Hkv][w_stride], or null for zeros
  float* w_out;
  int64_t w_stride;
  int32_t R;               // query rows of a KV head, 1..8
  int32_t parts, per_cta;  // CTAs per (sequence, KV head), and rounds of kAccPages pages of each
  int32_t vec;             // the accounts' rows are 16-byte aligned
};

// Row r's (m, 1 / l) over a sequence's group, by one warp: the merge of its partials, or what the
// attention kernel left for an unsplit group.
template <class MOf, class LOf>
__device__ __forceinline__ void row_stats(const AccountParams& p, const int4& g1, int seq, int head,
                                          int32_t Hkv, int r, int lane, float c2, MOf m_of,
                                          LOf l_of, float2* s_stats) {
  float2 st;
  if (g1.x > 1) {
    float M = -INFINITY, L = 0.f;
    for (int q = lane; q < g1.x; q += 32) {
      const float m = __ldcg(m_of(g1.y + q, head, r)), l = __ldcg(l_of(g1.y + q, head, r));
      if (m == -INFINITY) continue;
      const float top = fmaxf(M, m);
      L = L * fast_exp2((M - top) * c2) + l * fast_exp2((m - top) * c2);  // 0 while M is -inf
      M = top;
    }
    const float top = warp_max_f32(M);
    L = M == -INFINITY ? 0.f : L * fast_exp2((M - top) * c2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    st = make_float2(top, L > 0.f ? 1.f / L : 0.f);
  } else {
    st = p.stats[((int64_t)seq * Hkv + head) * p.R + r];
  }
  // a row that saw no key: its scores are -inf, and -inf - m must not be -inf + inf
  if (!(st.y > 0.f)) st.x = 0.f;
  if (lane == 0) s_stats[r] = st;
}

// One CTA's share: `unit` counts (sequence, KV head, part of the pages), parts innermost.
// A sequence's group (the one of this KV head) is groups[2 * group_of(seq, head)]; m_of and l_of give
// the address of row r's m and l in the group's partial q.
template <class GroupOf, class MOf, class LOf>
__device__ __forceinline__ void account_chunk(const AccountParams& p, const int4* groups,
                                              int32_t unit, int32_t Hkv, int32_t heads_per_group,
                                              float c2, GroupOf group_of, MOf m_of, LOf l_of) {
  __shared__ float2 s_stats[kAccRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = unit % p.parts, pair = unit / p.parts;
  const int head = pair % Hkv, seq = pair / Hkv;
  const int64_t group = group_of(seq, head);
  const int4 g0 = groups[2 * group], g1 = groups[2 * group + 1];  // written before the attention
  const int len = g0.w;
  const int first = part * p.per_cta * kAccPages;  // page
  // A sequence shorter than the longest has CTAs without pages. They end here, before the wait for
  // the attention kernel (the others, of which there is at least one, carry it to the next kernel).
  if ((int64_t)first * kPage >= len) return;  // uniform over the CTA
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int pages = min(p.per_cta * kAccPages, (len + kPage - 1) / kPage - first);
  const int key = 4 * (tid & 15);
  const float* src = p.scores + (((int64_t)g1.w + first + (tid >> 4)) * heads_per_group +
                                 (heads_per_group > 1 ? head : 0)) * p.R * kPage + key;
  const int64_t src_step = (int64_t)kAccPages * heads_per_group * p.R * kPage;
  int64_t t = (int64_t)(first + (tid >> 4)) * kPage + key;
  const int64_t row = ((int64_t)seq * Hkv + head) * p.w_stride;
  for (int done = 0; done < pages; done += kAccPages, src += src_step, t += kAccPages * kPage) {
    const bool real = t < len;
    // (the first page's scores are requested before the statistics are put together)
    float4 s[kAccRows];
#pragma unroll
    for (int r = 0; r < kAccRows; ++r)
      if (real && r < p.R) s[r] = __ldcs(reinterpret_cast<const float4*>(src + r * kPage));
    const int64_t at = row + t;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    if (real && p.w_in != nullptr) {
      if (p.vec) {
        const float4 v = *reinterpret_cast<const float4*>(p.w_in + at);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t + e < len) w[e] = p.w_in[at + e];
      }
    }
    if (done == 0) {
      if (warp < p.R) row_stats(p, g1, seq, head, Hkv, warp, lane, c2, m_of, l_of, s_stats);
      __syncthreads();
    }
    if (!real) break;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < kAccRows; ++r) {
      if (r >= p.R) break;
      const float2 st = s_stats[r];
      const float x[4] = {s[r].x, s[r].y, s[r].z, s[r].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = fmaf(fast_exp2((x[e] - st.x) * c2), st.y, sum[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] += sum[e];  // the account is rounded once per call
    if (p.vec && t + 4 <= len) {
      *reinterpret_cast<float4*>(p.w_out + at) = make_float4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (t + e < len) p.w_out[at + e] = w[e];
    }
  }
}

inline AccountParams account_params(const float* scores, const float2* stats, const float* w_in,
                                    float* w_out, int64_t w_stride, int32_t R,
                                    int32_t num_seqs, int32_t Hkv, int32_t max_seq_len,
                                    int64_t total_tokens, int32_t num_sms) {
  AccountParams a;
  a.scores = scores; a.stats = stats; a.w_in = w_in; a.w_out = w_out; a.w_stride = w_stride;
  a.R = R;
  // about one round of CTAs, each putting the statistics together once
  const int64_t rounds = (total_tokens / (kAccPages * kPage) + num_seqs) * Hkv;
  const int64_t places = (int64_t)kAccCtasPerSm * num_sms;
  const int64_t per = (rounds + places - 1) / places;
  a.per_cta = (int32_t)(per < 1 ? 1 : per > 64 ? 64 : per);
  const int64_t span = (int64_t)a.per_cta * kAccPages * kPage;
  a.parts = (int32_t)((max_seq_len + span - 1) / span);
  a.vec = w_stride % 4 == 0 && ((reinterpret_cast<uintptr_t>(w_in) |
                                 reinterpret_cast<uintptr_t>(w_out)) & 15u) == 0;
  return a;
}

// A merge-and-weights kernel as a programmatic dependent of the attention kernel before it.
template <class Kernel, class Merge>
cudaError_t launch_with_accounts(Kernel kernel, const Merge& mp, const AccountParams& a,
                                 int32_t merges, int64_t grid, cudaStream_t stream) {
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kAccThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, mp, a, merges);
}

}  // namespace kvnvfp4
