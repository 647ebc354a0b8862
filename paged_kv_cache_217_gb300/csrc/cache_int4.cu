// Cache operations of the 4-bit KV cache (int4_layout.cuh): the quantising
// write, the read of stored rows back to 16 bits, and the copy of blocks of a
// cache held in one pool.
//
// Write and read take one warp per (token, KV head): lane l holds D/32
// consecutive dims, so the 64 dims of a group sit in 2048/D neighbouring lanes
// whose minimum and maximum are joined by shuffles. Both are bound by bytes
// (4 D read and 9 D / 4 written per row pair, or the reverse).
#include <cuda_runtime.h>

#include <cstdint>

#include "device_common.cuh"
#include "int4_layout.cuh"
#include "launch.h"

namespace pkv {
namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <int BYTES>
struct Piece;  // a register of BYTES bytes
template <> struct Piece<1> { using type = unsigned char; };
template <> struct Piece<2> { using type = unsigned short; };
template <> struct Piece<4> { using type = uint32_t; };
template <> struct Piece<8> { using type = uint2; };
template <> struct Piece<16> { using type = uint4; };

// One lane's D/32 dims of a row quantised with its group, as packed codes
// (dim i in bits 4 i), and the group's {s, z}.
template <typename T, int D>
__device__ __forceinline__ uint32_t quantize_group(const T* xs, T& s_out, T& z_out) {
  constexpr int E = D / 32;
  float x[E], lo = INFINITY, hi = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    x[i] = to_f32<T>(xs[i]);
    bad |= !(fabsf(x[i]) < INFINITY);
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
  constexpr int LANES = kInt4Group / E;  // lanes of a group
#pragma unroll
  for (int m = 1; m < LANES; m <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(kFull, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, m));
  }
  const unsigned groups = __ballot_sync(kFull, bad);
  const unsigned mine = LANES == 32 ? kFull : ((1u << (LANES & 31)) - 1u) << ((threadIdx.x & 31) / LANES * LANES & 31);
  if (groups & mine) {
    s_out = z_out = from_f32<T>(NAN);
    return 0u;
  }
  s_out = from_f32<T>(__fdiv_rn(__fsub_rn(0.5f * hi, 0.5f * lo), 7.5f));
  z_out = from_f32<T>(lo);
  const float half_s = 0.5f * to_f32<T>(s_out), half_z = 0.5f * lo;
  uint32_t codes = 0;
  if (half_s > 0.f) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float c = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(0.5f * x[i], half_z), half_s)), 0.f), 15.f);
      codes |= uint32_t(c) << (4 * i);
    }
  }
  return codes;
}

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(T s, T z) {
  unsigned short a, b;
  memcpy(&a, &s, 2);
  memcpy(&b, &z, 2);
  return uint32_t(a) | (uint32_t(b) << 16);
}

template <typename T, int D>
__global__ void __launch_bounds__(256)
reshape_and_cache_int4_kernel(const T* __restrict__ k, const T* __restrict__ v, unsigned char* __restrict__ cache,
                              const int64_t* __restrict__ slots, int64_t rows, int num_kv_heads, int64_t num_slots,
                              unsigned int* status) {
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int E = D / 32;
  using In = typename Piece<2 * E>::type;
  const int64_t row = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;  // warp-uniform
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const int g = int(row % num_kv_heads);
  const int64_t t = row / num_kv_heads;
  const int64_t slot = __ldg(slots + t);
  const In kx = __ldg(reinterpret_cast<const In*>(k + row * D) + lane);
  const In vx = __ldg(reinterpret_cast<const In*>(v + row * D) + lane);
  if (slot < 0) return;
  if (slot >= num_slots) {
    if (g == 0 && lane == 0) flag(status, PKV_DEV_BAD_SLOT);
    return;
  }
  unsigned char* tile = cache + ((slot / kBlock) * num_kv_heads + g) * kv4_tile_bytes(D);
  const int r = int(slot % kBlock);
  T ks, kz, vs, vz;
  const uint32_t kc = quantize_group<T, D>(reinterpret_cast<const T*>(&kx), ks, kz);
  const uint32_t vc = quantize_group<T, D>(reinterpret_cast<const T*>(&vx), vs, vz);
  using Out = typename Piece<E / 2>::type;
  constexpr int LPW = 8 / E;  // lanes of one word
  const int w = lane / LPW, sub = (lane % LPW) * (E / 2);
  *reinterpret_cast<Out*>(tile + kv4_k_word<D>(r, w) + sub) = Out(kc);
  *reinterpret_cast<Out*>(tile + kv4_v_word<D>(r, w) + sub) = Out(vc);
  constexpr int LANES = kInt4Group / E;
  if (lane % LANES == 0) {
    *reinterpret_cast<uint32_t*>(tile + kv4_k_pair<D>(r, lane / LANES)) = pack_pair<T>(ks, kz);
    *reinterpret_cast<uint32_t*>(tile + kv4_v_pair<D>(r, lane / LANES)) = pack_pair<T>(vs, vz);
  }
}

// One lane's D/32 dims of a stored row, rounded once to T.
template <typename T, int D>
__device__ __forceinline__ typename Piece<D / 16>::type read_group(uint32_t codes, uint32_t pair) {
  constexpr int E = D / 32;
  typename Piece<2 * E>::type out;
  T* o = reinterpret_cast<T*>(&out);
  unsigned short a = (unsigned short)(pair & 0xffffu), b = (unsigned short)(pair >> 16);
  T s, z;
  memcpy(&s, &a, 2);
  memcpy(&z, &b, 2);
  const float sf = to_f32<T>(s), zf = to_f32<T>(z);
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = from_f32<T>(fmaf(float((codes >> (4 * i)) & 15u), sf, zf));
  return out;
}

template <typename T, int D>
__global__ void __launch_bounds__(256)
gather_cache_int4_kernel(T* __restrict__ k, T* __restrict__ v, const unsigned char* __restrict__ cache,
                         const int64_t* __restrict__ slots, int64_t rows, int num_kv_heads, int64_t num_slots,
                         unsigned int* status) {
  constexpr int E = D / 32;
  using Row = typename Piece<2 * E>::type;
  using In = typename Piece<E / 2>::type;
  const int64_t row = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const int g = int(row % num_kv_heads);
  const int64_t slot = __ldg(slots + row / num_kv_heads);
  Row kx{}, vx{};
  if (slot >= num_slots) {
    if (g == 0 && lane == 0) flag(status, PKV_DEV_BAD_SLOT);
  } else if (slot >= 0) {
    const unsigned char* tile = cache + ((slot / kBlock) * num_kv_heads + g) * kv4_tile_bytes(D);
    const int r = int(slot % kBlock);
    constexpr int LPW = 8 / E, LANES = kInt4Group / E;
    const int w = lane / LPW, sub = (lane % LPW) * (E / 2);
    const uint32_t kc = *reinterpret_cast<const In*>(tile + kv4_k_word<D>(r, w) + sub);
    const uint32_t vc = *reinterpret_cast<const In*>(tile + kv4_v_word<D>(r, w) + sub);
    const uint32_t kp = *reinterpret_cast<const uint32_t*>(tile + kv4_k_pair<D>(r, lane / LANES));
    const uint32_t vp = *reinterpret_cast<const uint32_t*>(tile + kv4_v_pair<D>(r, lane / LANES));
    kx = read_group<T, D>(kc, kp);
    vx = read_group<T, D>(vc, vp);
  }
  reinterpret_cast<Row*>(k + row * D)[lane] = kx;
  reinterpret_cast<Row*>(v + row * D)[lane] = vx;
}

constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;

__global__ void __launch_bounds__(kCopyThreads)
copy_blocks_pool_kernel(uint4* __restrict__ pool, const int64_t* __restrict__ pairs, int64_t vec_per_block,
                        int num_blocks, unsigned int* status) {
  const int64_t src = __ldg(pairs + 2 * int64_t(blockIdx.y)), dst = __ldg(pairs + 2 * int64_t(blockIdx.y) + 1);
  if (src == -1 && dst == -1) return;  // padding of a fixed-size list
  if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag(status, PKV_DEV_BAD_PAIR);
    return;
  }
  const int64_t base = int64_t(blockIdx.x) * kCopyThreads * kCopyVecs + threadIdx.x;
  uint4 x[kCopyVecs];
#pragma unroll
  for (int u = 0; u < kCopyVecs; ++u) {
    const int64_t i = base + u * kCopyThreads;
    if (i < vec_per_block) x[u] = pool[src * vec_per_block + i];
  }
#pragma unroll
  for (int u = 0; u < kCopyVecs; ++u) {
    const int64_t i = base + u * kCopyThreads;
    if (i < vec_per_block) pool[dst * vec_per_block + i] = x[u];
  }
}

template <typename T, int D>
cudaError_t write_or_gather(bool gather, void* k, void* v, void* cache, const int64_t* slots, int64_t rows,
                            int num_kv_heads, int64_t num_slots, unsigned int* status, cudaStream_t stream) {
  const unsigned ctas = unsigned((rows + 7) / 8);  // 8 warps (rows) per CTA
  if (gather)
    gather_cache_int4_kernel<T, D><<<ctas, 256, 0, stream>>>(static_cast<T*>(k), static_cast<T*>(v),
                                                             static_cast<const unsigned char*>(cache), slots, rows,
                                                             num_kv_heads, num_slots, status);
  else
    reshape_and_cache_int4_kernel<T, D><<<ctas, 256, 0, stream>>>(static_cast<const T*>(k), static_cast<const T*>(v),
                                                                  static_cast<unsigned char*>(cache), slots, rows,
                                                                  num_kv_heads, num_slots, status);
  return cudaGetLastError();
}

template <typename T>
cudaError_t write_or_gather_t(bool gather, void* k, void* v, void* cache, const int64_t* slots, int64_t rows,
                              int num_kv_heads, int head_dim, int64_t num_slots, unsigned int* status,
                              cudaStream_t stream) {
  switch (head_dim) {
    case 64: return write_or_gather<T, 64>(gather, k, v, cache, slots, rows, num_kv_heads, num_slots, status, stream);
    case 128: return write_or_gather<T, 128>(gather, k, v, cache, slots, rows, num_kv_heads, num_slots, status, stream);
    case 256: return write_or_gather<T, 256>(gather, k, v, cache, slots, rows, num_kv_heads, num_slots, status, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_cache_int4(bool gather, void* k, void* v, bool bf16, void* cache, const int64_t* slots,
                              int num_tokens, int num_kv_heads, int head_dim, int num_blocks, unsigned int* status,
                              cudaStream_t stream) {
  const int64_t rows = int64_t(num_tokens) * num_kv_heads, num_slots = int64_t(num_blocks) * kBlock;
  return bf16 ? write_or_gather_t<__nv_bfloat16>(gather, k, v, cache, slots, rows, num_kv_heads, head_dim, num_slots,
                                                 status, stream)
              : write_or_gather_t<__half>(gather, k, v, cache, slots, rows, num_kv_heads, head_dim, num_slots, status,
                                          stream);
}

cudaError_t launch_copy_blocks_pool(void* pool, const int64_t* pairs, int num_pairs, int64_t bytes_per_block,
                                    int num_blocks, unsigned int* status, cudaStream_t stream) {
  const int64_t vecs = bytes_per_block / 16, per_cta = kCopyThreads * kCopyVecs;
  const dim3 grid(unsigned((vecs + per_cta - 1) / per_cta), unsigned(num_pairs));
  copy_blocks_pool_kernel<<<grid, kCopyThreads, 0, stream>>>(static_cast<uint4*>(pool), pairs, vecs, num_blocks,
                                                             status);
  return cudaGetLastError();
}

}  // namespace pkv
