// Latent attention over a paged cache of one shared row per token: the cache
// write, and the launch of the decode (latent_decode.cuh).
#include <cuda_runtime.h>

#include <cstdint>

#include "decode_launch.cuh"
#include "latent_decode.cuh"
#include "launch.h"

namespace pkv {
namespace {

// One thread per 16-byte vector of a row: the latent part, then the rotary part.
__global__ void __launch_bounds__(256)
latent_write_kernel(const uint4* __restrict__ latent, const uint4* __restrict__ rope, uint4* __restrict__ cache,
                    const int64_t* __restrict__ slots, int64_t total, int64_t latent_stride, int64_t rope_stride,
                    int64_t num_slots, unsigned int* status) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= total) return;
  constexpr int VECS = kLatentRow / 8;
  const int64_t t = i / VECS;
  const int c = int(i % VECS);
  const int64_t slot = __ldg(slots + t);
  const uint4 x = c < kLatentDim / 8 ? __ldg(latent + t * latent_stride + c)
                                     : __ldg(rope + t * rope_stride + c - kLatentDim / 8);
  if (slot < 0) return;
  if (slot >= num_slots) {
    if (c == 0) flag(status, PKV_DEV_BAD_SLOT);
    return;
  }
  cache[slot * VECS + c] = x;
}

// Heads per CTA: all of them in blocks of at most 64, evenly.
struct LatentShape {
  int blocks, heads, n, ranges;
};
LatentShape latent_shape(int num_seqs, int num_heads, int max_blocks_per_seq) {
  LatentShape p;
  p.blocks = (num_heads + 63) / 64;
  p.heads = (num_heads + p.blocks - 1) / p.blocks;
  p.n = p.heads <= 16 ? 16 : p.heads <= 32 ? 32 : 64;
  const int64_t tiles =
      int64_t(num_seqs) * ((int64_t(max_blocks_per_seq) * kBlock + kLatentTile - 1) / kLatentTile);
  p.ranges = kLatentSms / p.blocks > 0 ? kLatentSms / p.blocks : 1;
  if (tiles < p.ranges) p.ranges = int(tiles);
  return p;
}

template <typename T, int N>
cudaError_t launch_n(LatentArgs a, const LatentShape& p, const CUtensorMap& cache_map, const CUtensorMap& q_map,
                     cudaStream_t stream) {
  using C = LatentCfg<N>;
  static bool configured[kMaxDevices] = {};
  cudaError_t err = configure_once(latent_decode_kernel<T, N>, C::SMEM_BYTES, configured);
  if (err != cudaSuccess) return err;
  err = launch_pdl(latent_decode_kernel<T, N>, dim3(unsigned(p.blocks * p.ranges)), dim3(kLatentThreads), C::SMEM_BYTES,
                   stream, a, cache_map, q_map);
  if (err != cudaSuccess) return err;
  if (p.ranges == 1) return cudaSuccess;  // one range: nothing crosses
  const unsigned items = unsigned(a.desc_by_seq ? a.num_seqs : p.ranges), heads = unsigned(a.num_heads);
  // Few heads to join, of many pieces each: 4 CTAs a head. Whole calls, Z = 4 against
  // 1: 64 heads of one long sequence 37.5 us, 65.1; 4 sequences x 16 heads 19.4,
  // 25.6; x 128 heads 40.9, 33.0; 96 sequences x 16 heads 78, 48.
  if (int64_t(items) * heads <= 2 * kLatentSms)
    return launch_pdl(latent_merge_kernel<T, N, 4>, dim3(items, heads, 4), dim3(256), 0, stream, a);
  return launch_pdl(latent_merge_kernel<T, N, 1>, dim3(items, (heads + 1) / 2), dim3(256), 0, stream, a);
}

template <typename T>
cudaError_t launch_t(LatentArgs a, const CUtensorMap& cache_map, const CUtensorMap& q_map, cudaStream_t stream) {
  const LatentShape p = latent_shape(a.num_seqs, a.num_heads, a.max_blocks_per_seq);
  a.ranges = p.ranges;
  a.head_blocks = p.blocks;
  a.block_heads = p.heads;
  a.desc_by_seq = a.num_seqs <= p.ranges;
  a.desc = static_cast<int2*>(a.workspace);
  a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(a.workspace) + latent_desc_bytes(p.ranges));
  a.part_o = reinterpret_cast<float*>(a.part_ml + size_t(2) * p.ranges * p.blocks * p.n);
  switch (p.n) {
    case 16: return launch_n<T, 16>(a, p, cache_map, q_map, stream);
    case 32: return launch_n<T, 32>(a, p, cache_map, q_map, stream);
    default: return launch_n<T, 64>(a, p, cache_map, q_map, stream);
  }
}

}  // namespace

cudaError_t launch_latent_write(const void* latent, const void* rope, void* cache, const int64_t* slots,
                                int num_tokens, int64_t latent_stride, int64_t rope_stride, int num_blocks,
                                unsigned int* status, cudaStream_t stream) {
  const int64_t total = int64_t(num_tokens) * (kLatentRow / 8);
  latent_write_kernel<<<unsigned((total + 255) / 256), 256, 0, stream>>>(
      static_cast<const uint4*>(latent), static_cast<const uint4*>(rope), static_cast<uint4*>(cache), slots, total,
      latent_stride / 8, rope_stride / 8, int64_t(num_blocks) * kBlock, status);
  return cudaGetLastError();
}

// Range descriptors, then per range two partial results of every head: (max,
// sum) pairs and fp32 accumulators.
size_t latent_workspace_bytes(int num_seqs, int num_heads, int max_blocks_per_seq) {
  const LatentShape p = latent_shape(num_seqs, num_heads, max_blocks_per_seq);
  return latent_desc_bytes(p.ranges) +
         size_t(2) * p.ranges * p.blocks * p.n * (sizeof(float2) + kLatentDim * sizeof(float));
}

int latent_query_box(int num_seqs, int num_heads, int max_blocks_per_seq) {
  return latent_shape(num_seqs, num_heads, max_blocks_per_seq).n;
}

cudaError_t launch_latent_decode(const LatentArgs& a, bool bf16, const CUtensorMap& cache_map,
                                 const CUtensorMap& q_map, cudaStream_t stream) {
  return bf16 ? launch_t<__nv_bfloat16>(a, cache_map, q_map, stream) : launch_t<__half>(a, cache_map, q_map, stream);
}

}  // namespace pkv
