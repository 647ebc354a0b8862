// Launch of the prompt, cross and shared-prefix attention kernels (prompt.cuh).
#include <cuda_runtime.h>

#include <cstdint>

#include "decode_launch.cuh"
#include "launch.h"
#include "prompt.cuh"

namespace pkv {
namespace {

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

struct PromptShape {
  int tile_tokens, block_tokens, shares;
  size_t slot_rows, rows;  // rows of a slot; of items that are not cut but kept all the same (prefix decode)
};

PromptShape prompt_shape(const PromptArgs& a, int head_dim) {
  PromptShape p;
  const int groups = head_dim == 256 ? 1 : 2, tile = head_dim == 256 ? 64 : 128;
  p.tile_tokens = prompt_tile_tokens(a.num_q_heads / a.num_kv_heads);
  p.block_tokens = p.tile_tokens * groups;
  p.slot_rows = a.num_tokens > p.tile_tokens ? size_t(128) * groups : 128;
  p.rows = a.query_starts ? 0 : size_t(2) * a.num_seqs * a.num_q_heads;
  // no more shares than tiles
  const int64_t blocks = int64_t(a.num_tokens) / p.block_tokens + a.num_seqs + (a.num_groups ? a.num_seqs : 0);
  const int64_t tiles = blocks * a.num_kv_heads * ((int64_t(a.max_blocks_per_seq) * kBlock + tile - 1) / tile + 1);
  p.shares = tiles < kPromptSms ? int(tiles) : kPromptSms;
  return p;
}

template <typename T, int D>
cudaError_t launch_d(const PromptArgs& a, const PromptMaps& maps, cudaStream_t stream) {
  using C = PromptCfg<D>;
  static bool configured[kMaxDevices] = {};
  cudaError_t err = configure_once(prompt_kernel<T, D>, C::SMEM_BYTES, configured);
  if (err != cudaSuccess) return err;
  err = launch_pdl(prompt_kernel<T, D>, dim3(unsigned(a.shares)), dim3(C::THREADS), C::SMEM_BYTES, stream, a, maps.q,
                   maps.q1, maps.k, maps.v);
  if (err != cudaSuccess) return err;
  if (!a.query_starts)
    return launch_pdl(prefix_join_kernel<T, D>, dim3(unsigned((int64_t(a.num_seqs) * a.num_q_heads + 7) / 8)), dim3(256), 0,
                      stream, a);
  if (a.shares == 1) return cudaSuccess;  // nothing is cut
  return launch_pdl(prompt_join_kernel<T, D>, dim3(unsigned(a.shares), 8), dim3(256), 0, stream, a);
}

template <typename T>
cudaError_t launch_t(const PromptArgs& a, int head_dim, const PromptMaps& maps, cudaStream_t stream) {
  if (head_dim == 64) return launch_d<T, 64>(a, maps, stream);
  if (head_dim == 128) return launch_d<T, 128>(a, maps, stream);
  return launch_d<T, 256>(a, maps, stream);
}

}  // namespace

// Per share: what is cut; per item (prefix decode): where its pieces are; then (maximum,
// sum) pairs and fp32 accumulators of two slots a share and of kept rows.
size_t prompt_workspace_bytes(const PromptArgs& a, int head_dim) {
  const PromptShape p = prompt_shape(a, head_dim);
  const size_t links = a.query_starts ? size_t(p.shares) * sizeof(int4) : size_t(2) * a.num_seqs * a.num_kv_heads * sizeof(int2);
  return round16(links) + round16(size_t(p.shares) * sizeof(int)) +
         (p.slot_rows * 2 * p.shares + p.rows) * (sizeof(float2) + size_t(head_dim) * sizeof(float));
}

cudaError_t launch_prompt(PromptArgs a, bool bf16, int head_dim, void* workspace, const PromptMaps& maps,
                          cudaStream_t stream) {
  const PromptShape p = prompt_shape(a, head_dim);
  a.tile_tokens = p.tile_tokens;
  a.block_tokens = p.block_tokens;
  a.shares = p.shares;
  a.slot_rows = p.slot_rows;
  char* at = static_cast<char*>(workspace);
  a.desc = reinterpret_cast<int4*>(at);
  a.link = reinterpret_cast<int2*>(at);
  at += round16(a.query_starts ? size_t(p.shares) * sizeof(int4) : size_t(2) * a.num_seqs * a.num_kv_heads * sizeof(int2));
  a.more = reinterpret_cast<int*>(at);
  at += round16(size_t(p.shares) * sizeof(int));
  a.part_o = reinterpret_cast<float*>(at);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (p.slot_rows * 2 * p.shares + p.rows) * head_dim);
  return bf16 ? launch_t<__nv_bfloat16>(a, head_dim, maps, stream) : launch_t<__half>(a, head_dim, maps, stream);
}

}  // namespace pkv
