// Attention of several query tokens per sequence over the paged cache, and decode
// attention of groups that share a prefix: the plain form, a warp per (token, head).
#include <cuda_runtime.h>

#include <cstdint>

#include "device_common.cuh"
#include "launch.h"

namespace pkv {
namespace {

template <typename T, int D>
__global__ void __launch_bounds__(128) prompt_rows_kernel(const PromptArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) {
    const int32_t* starts = a.num_groups ? a.group_starts : a.query_starts;
    const int n = a.num_groups ? a.num_groups : starts ? a.num_seqs : -1, most = a.num_tokens;
    for (int i = threadIdx.x; i <= n; i += 128)
      if (starts[i] < 0 || starts[i] > most || (i && starts[i] < starts[i - 1])) flag(a.status, PKV_DEV_BAD_START);
  }
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= int64_t(a.num_tokens) * a.num_q_heads) return;
  const int t = int(row / a.num_q_heads), h = int(row % a.num_q_heads), g = h / a.group;
  auto last_at = [&](const int32_t* starts, int n, int x) {  // largest i < n with starts[i] <= x, or -1
    int lo = -1, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (starts[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  int s = t, n = 1, place = 0;
  if (a.query_starts) {
    s = last_at(a.query_starts, a.num_seqs, t);
    if (s < 0) return;
    const int end = min(a.query_starts[s + 1], a.num_tokens);
    if (t >= end) return;
    n = end - a.query_starts[s];
    place = t - a.query_starts[s];
  }
  const int most = a.max_blocks_per_seq * kBlock, raw = a.context_lens[s];
  if ((raw < 0 || raw > most) && lane == 0) flag(a.status, PKV_DEV_BAD_CONTEXT_LEN);
  const int L = raw < 0 ? 0 : raw > most ? most : raw;
  const int hi = a.causal ? min(L, L - n + place + 1) : L;
  const int lo = a.window ? max(0, hi - a.window) : 0;
  int shared = 0, leader = s;
  if (a.num_groups) {
    const int i = last_at(a.group_starts, a.num_groups, s);
    if (i >= 0 && s < a.group_starts[i + 1]) {
      leader = min(max(a.group_starts[i], 0), a.num_seqs - 1);
      shared = min(max(a.prefix_blocks[i], 0), a.max_blocks_per_seq);
    }
  }
  const T* q = static_cast<const T*>(a.q) + row * D;
  float qf[E], acc[E] = {};
  for (int e = 0; e < E; ++e) qf[e] = float(q[lane + 32 * e]) * a.scale_log2;
  float m = -INFINITY, l = 0.f;
  for (int p = lo; p < hi; ++p) {
    int id = a.block_tables[size_t(p / kBlock < shared ? leader : s) * a.max_blocks_per_seq + p / kBlock];
    if (id < 0 || id >= a.num_blocks) {
      if (lane == 0) flag(a.status, PKV_DEV_BAD_BLOCK_ID);
      id = 0;
    }
    const size_t at = ((size_t(id) * a.num_kv_heads + g) * kBlock + p % kBlock) * D;
    float x = 0.f;
    for (int e = 0; e < E; ++e) x += qf[e] * float(static_cast<const T*>(a.k_pool)[at + lane + 32 * e]);
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    const float now = fmaxf(m, x), back = now == -INFINITY ? 1.f : exp2f(m - now);
    const float w = now == -INFINITY ? 0.f : exp2f(x - now);
    m = now;
    l = l * back + w;
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * back + w * float(static_cast<const T*>(a.v_pool)[at + lane + 32 * e]);
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  for (int e = 0; e < E; ++e) static_cast<T*>(a.out)[row * D + lane + 32 * e] = T(acc[e] * inv);
}

template <typename T>
cudaError_t launch_t(const PromptArgs& a, int head_dim, cudaStream_t stream) {
  const unsigned grid = unsigned((int64_t(a.num_tokens) * a.num_q_heads + 3) / 4);
  if (head_dim == 64) prompt_rows_kernel<T, 64><<<grid, 128, 0, stream>>>(a);
  else if (head_dim == 128) prompt_rows_kernel<T, 128><<<grid, 128, 0, stream>>>(a);
  else prompt_rows_kernel<T, 256><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs& a, bool bf16, int head_dim, cudaStream_t stream) {
  return bf16 ? launch_t<__nv_bfloat16>(a, head_dim, stream) : launch_t<__half>(a, head_dim, stream);
}

}  // namespace pkv
