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
  const int groups = head_dim == 256 ? 1 : 2;
  p.tile_tokens = prompt_tile_tokens(a.num_q_heads / a.num_kv_heads);
  p.block_tokens = p.tile_tokens * groups;
  p.slot_rows = a.num_tokens > p.tile_tokens ? size_t(128) * groups : 128;
  p.rows = a.query_starts ? 0 : size_t(2) * a.num_seqs * a.num_q_heads;
  const int64_t blocks = int64_t(a.num_tokens) / p.block_tokens + a.num_groups + a.num_seqs;
  constexpr int kShare = kPromptShareTiles * kPromptTile;
  const int64_t most = blocks * a.num_kv_heads * ((int64_t(a.max_blocks_per_seq) * kBlock + kShare - 1) / kShare + 1);
  p.shares = most < kPromptSms ? int(most) : kPromptSms;
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
    return launch_pdl(a.tails ? prefix_join_kernel<T, D, true> : prefix_join_kernel<T, D, false>, dim3(unsigned((int64_t(a.num_seqs) * a.num_q_heads + 7) / 8)), dim3(256), 0,
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

namespace {
// Per share: what is cut; per item (prefix decode): where its pieces are; whether shares begin
// inside an item; where prefixes end; what the decode grid takes; then fp32 accumulators and (maximum, sum) pairs of two
// slots a share and of kept rows.
size_t lay_out(PromptArgs* a, int head_dim, char* workspace) {
  const PromptShape p = prompt_shape(*a, head_dim);
  a->tile_tokens = p.tile_tokens;
  a->block_tokens = p.block_tokens;
  a->shares = p.shares;
  a->slot_rows = p.slot_rows;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* const here = workspace + at;
    at += round16(bytes);
    return here;
  };
  char* const links = take(a->query_starts ? size_t(p.shares) * sizeof(int4) : size_t(2) * a->num_seqs * a->num_kv_heads * sizeof(int2));
  a->desc = reinterpret_cast<int4*>(links);
  a->link = reinterpret_cast<int2*>(links);
  a->more = reinterpret_cast<int*>(take(size_t(p.shares) * sizeof(int)));
  a->from = reinterpret_cast<int32_t*>(take(size_t(a->num_seqs) * sizeof(int32_t)));
  a->limit = reinterpret_cast<int*>(take(sizeof(int)));
  const size_t rows = p.slot_rows * 2 * p.shares + p.rows;
  a->part_o = reinterpret_cast<float*>(take(rows * head_dim * sizeof(float)));
  a->part_ml = reinterpret_cast<float2*>(take(rows * sizeof(float2)));
  return at;
}
}  // namespace

size_t prompt_workspace_bytes(const PromptArgs& a, int head_dim) {
  PromptArgs b = a;
  return lay_out(&b, head_dim, nullptr);
}

PromptTails prompt_tails(PromptArgs a, int head_dim, void* workspace) {
  lay_out(&a, head_dim, static_cast<char*>(workspace));
  const size_t kept = a.slot_rows * 2 * a.shares;
  return {a.limit, a.from, a.part_ml + kept, a.part_o + kept * head_dim};
}

cudaError_t launch_prompt(PromptArgs a, bool bf16, int head_dim, void* workspace, const PromptMaps& maps,
                          cudaStream_t stream) {
  lay_out(&a, head_dim, static_cast<char*>(workspace));
  return bf16 ? launch_t<__nv_bfloat16>(a, head_dim, maps, stream) : launch_t<__half>(a, head_dim, maps, stream);
}

}  // namespace pkv
