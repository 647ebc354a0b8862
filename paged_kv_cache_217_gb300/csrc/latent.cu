// Latent attention over a paged cache of one shared row per token: the cache
// write and the decode (absorbed form). The decode here is a plain kernel that
// is right for every case (one CTA per (sequence, 8 heads), CUDA-core
// products).
#include <cuda_runtime.h>

#include <cstdint>

#include "device_common.cuh"
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

constexpr int kHeads = 8;
constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads) latent_decode_kernel(const LatentArgs a) {
  extern __shared__ float sm[];
  float(*rows)[kLatentRow + 1] = reinterpret_cast<float(*)[kLatentRow + 1]>(sm);
  float(*qs)[kLatentRow] = reinterpret_cast<float(*)[kLatentRow]>(sm + kBlock * (kLatentRow + 1));
  __shared__ float x[kHeads][kBlock], part[2][kHeads][kBlock], mrun[kHeads], lrun[kHeads], alpha[kHeads];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int s = blockIdx.y, h0 = blockIdx.x * kHeads, tid = threadIdx.x;
  const int heads = min(kHeads, a.num_heads - h0);
  int L = a.context_lens[s];
  const int max_len = a.max_blocks_per_seq * kBlock;
  if (L < 0 || L > max_len) {
    if (tid == 0 && h0 == 0) flag(a.status, PKV_DEV_BAD_CONTEXT_LEN);
    L = L < 0 ? 0 : max_len;
  }
  const T* q = static_cast<const T*>(a.q) + (size_t(s) * a.num_heads + h0) * kLatentRow;
  for (int i = tid; i < heads * kLatentRow; i += kThreads)
    qs[i / kLatentRow][i % kLatentRow] = float(q[i]) * a.scale_log2;
  if (tid < kHeads) mrun[tid] = -INFINITY, lrun[tid] = 0.f;
  float acc[kHeads][2] = {};
  for (int t0 = 0; t0 < L; t0 += kBlock) {
    int id = a.block_tables[size_t(s) * a.max_blocks_per_seq + t0 / kBlock];
    if (id < 0 || id >= a.num_blocks) {
      if (tid == 0) flag(a.status, PKV_DEV_BAD_BLOCK_ID);
      id = 0;
    }
    __syncthreads();
    const T* src = static_cast<const T*>(a.cache) + size_t(id) * kBlock * kLatentRow;
    for (int i = tid; i < kBlock * kLatentRow; i += kThreads) {
      const int r = i / kLatentRow;
      rows[r][i % kLatentRow] = t0 + r < L ? float(src[i]) : 0.f;
    }
    __syncthreads();
    {
      const int half = tid / 128, h = tid % 128 / kBlock, r = tid % kBlock;
      float dot = 0.f;
      if (h < heads)
        for (int d = half * (kLatentRow / 2); d < (half + 1) * (kLatentRow / 2); ++d) dot = fmaf(qs[h][d], rows[r][d], dot);
      part[half][h][r] = dot;
    }
    __syncthreads();
    if (tid < heads) {
      float m = mrun[tid];
      for (int r = 0; r < kBlock; ++r) {
        x[tid][r] = t0 + r < L ? part[0][tid][r] + part[1][tid][r] : -INFINITY;
        m = fmaxf(m, x[tid][r]);
      }
      const float ref = m == -INFINITY ? 0.f : m;
      alpha[tid] = fast_exp2(mrun[tid] - ref);
      float l = lrun[tid] * alpha[tid];
      for (int r = 0; r < kBlock; ++r) {
        x[tid][r] = fast_exp2(x[tid][r] - ref);
        l += x[tid][r];
      }
      mrun[tid] = m;
      lrun[tid] = l;
    }
    __syncthreads();
    for (int h = 0; h < heads; ++h) {
      float o0 = acc[h][0] * alpha[h], o1 = acc[h][1] * alpha[h];
      for (int r = 0; r < kBlock; ++r) {
        o0 = fmaf(x[h][r], rows[r][tid], o0);
        o1 = fmaf(x[h][r], rows[r][tid + kThreads], o1);
      }
      acc[h][0] = o0;
      acc[h][1] = o1;
    }
  }
  __syncthreads();
  T* out = static_cast<T*>(a.out) + (size_t(s) * a.num_heads + h0) * kLatentDim;
  for (int h = 0; h < heads; ++h) {
    const float inv = L == 0 ? 0.f : 1.f / lrun[h];
    out[h * kLatentDim + tid] = T(acc[h][0] * inv);
    out[h * kLatentDim + tid + kThreads] = T(acc[h][1] * inv);
  }
}

template <typename T>
cudaError_t launch_t(const LatentArgs& a, cudaStream_t stream) {
  const size_t smem = (size_t(kBlock) * (kLatentRow + 1) + kHeads * kLatentRow) * sizeof(float);
  cudaError_t err = cudaFuncSetAttribute(latent_decode_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (err != cudaSuccess) return err;
  latent_decode_kernel<T><<<dim3(unsigned((a.num_heads + kHeads - 1) / kHeads), unsigned(a.num_seqs)), kThreads, smem,
                            stream>>>(a);
  return cudaGetLastError();
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

size_t latent_workspace_bytes(int, int, int) { return 0; }

cudaError_t launch_latent_decode(const LatentArgs& a, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_t<__nv_bfloat16>(a, stream) : launch_t<__half>(a, stream);
}

}  // namespace pkv
