// Decode attention over the 4-bit KV cache: a plain kernel that is right for
// every case (one CTA per (sequence, KV head), tiles dequantised to fp32 in
// shared memory, CUDA-core products).
#include <cuda_runtime.h>

#include <cstdint>

#include "decode.cuh"
#include "int4_layout.cuh"
#include "launch.h"

namespace pkv {
namespace {

template <typename T, int D>
__global__ void __launch_bounds__(256) paged_decode_int4_kernel(const DecodeArgs a) {
  __shared__ __align__(16) unsigned char raw[kv4_tile_bytes(D)];
  __shared__ float kf[kBlock][D + 1], vf[kBlock][D], qs[8][D], x[8][kBlock];
  __shared__ float mrun[8], lrun[8], alpha[8];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int g = blockIdx.x, s = long_first_seq<8>(a, blockIdx.y), tid = threadIdx.x;
  const int hq0 = g * a.group;
  int L = a.context_lens[s];
  const int max_len = a.max_blocks_per_seq * kBlock;
  if (L < 0 || L > max_len) {
    if (tid == 0 && g == 0) flag(a.status, PKV_DEV_BAD_CONTEXT_LEN);
    L = L < 0 ? 0 : max_len;
  }
  const TokenRange tr = token_range(L, a.window);
  const T* q = static_cast<const T*>(a.q) + (size_t(s) * a.num_q_heads + hq0) * D;
  for (int i = tid; i < a.group * D; i += 256) qs[i / D][i % D] = float(q[i]) * a.scale_log2;
  if (tid < 8) mrun[tid] = -INFINITY, lrun[tid] = 0.f;
  float acc[8 * D / 256];
#pragma unroll
  for (int i = 0; i < 8 * D / 256; ++i) acc[i] = 0.f;
  const unsigned char* cache = static_cast<const unsigned char*>(a.k_pool);
  for (int t0 = tr.aligned; t0 < L; t0 += kBlock) {
    int id = a.block_tables[size_t(s) * a.max_blocks_per_seq + t0 / kBlock];
    if (id < 0 || id >= a.num_blocks) {
      if (tid == 0) flag(a.status, PKV_DEV_BAD_BLOCK_ID);
      id = 0;
    }
    __syncthreads();
    const uint4* src = reinterpret_cast<const uint4*>(cache + (size_t(id) * a.num_kv_heads + g) * kv4_tile_bytes(D));
    for (int i = tid; i < kv4_tile_bytes(D) / 16; i += 256) reinterpret_cast<uint4*>(raw)[i] = src[i];
    __syncthreads();
    for (int i = tid; i < kBlock * D; i += 256) {
      const int r = i / D, d = i % D;
      const bool live = t0 + r >= tr.first && t0 + r < L;
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(raw + kv4_k_word<D>(r, d / 8));
      const uint32_t vw = *reinterpret_cast<const uint32_t*>(raw + kv4_v_word<D>(r, d / 8));
      const T* kp = reinterpret_cast<const T*>(raw + kv4_k_pair<D>(r, d / kInt4Group));
      const T* vp = reinterpret_cast<const T*>(raw + kv4_v_pair<D>(r, d / kInt4Group));
      kf[r][d] = live ? fmaf(float((kw >> (4 * (d % 8))) & 15u), float(kp[0]), float(kp[1])) : 0.f;
      vf[r][d] = live ? fmaf(float((vw >> (4 * (d % 8))) & 15u), float(vp[0]), float(vp[1])) : 0.f;
    }
    __syncthreads();
    if (tid < 8 * kBlock && tid / kBlock < a.group) {
      const int h = tid / kBlock, r = tid % kBlock;
      float dot = 0.f;
      for (int d = 0; d < D; ++d) dot = fmaf(qs[h][d], kf[r][d], dot);
      x[h][r] = t0 + r >= tr.first && t0 + r < L ? dot : -INFINITY;
    }
    __syncthreads();
    if (tid < a.group) {
      float m = mrun[tid];
      for (int r = 0; r < kBlock; ++r) m = fmaxf(m, x[tid][r]);
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
#pragma unroll
    for (int i = 0; i < 8 * D / 256; ++i) {
      const int e = tid + 256 * i, h = e / D, d = e % D;
      if (h >= a.group) continue;
      float o = acc[i] * alpha[h];
      for (int r = 0; r < kBlock; ++r) o = fmaf(x[h][r], vf[r][d], o);
      acc[i] = o;
    }
  }
  __syncthreads();
  T* out = static_cast<T*>(a.out) + (size_t(s) * a.num_q_heads + hq0) * D;
#pragma unroll
  for (int i = 0; i < 8 * D / 256; ++i) {
    const int e = tid + 256 * i;
    if (e / D < a.group) out[e] = T(L == 0 ? 0.f : acc[i] / lrun[e / D]);
  }
}

template <typename T>
cudaError_t launch_t(const DecodeArgs& a, int head_dim, cudaStream_t stream) {
  const dim3 grid(unsigned(a.num_kv_heads), unsigned(a.num_seqs));
  switch (head_dim) {
    case 64: paged_decode_int4_kernel<T, 64><<<grid, 256, 0, stream>>>(a); break;
    case 128: paged_decode_int4_kernel<T, 128><<<grid, 256, 0, stream>>>(a); break;
    case 256: paged_decode_int4_kernel<T, 256><<<grid, 256, 0, stream>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_int4(const DecodeArgs& a, bool bf16, int head_dim, int gpad, cudaStream_t stream) {
  (void)gpad;
  return bf16 ? launch_t<__nv_bfloat16>(a, head_dim, stream) : launch_t<__half>(a, head_dim, stream);
}

}  // namespace pkv
