// Cache operations of the 4-bit KV cache (int4_layout.cuh): the quantising
// write, the read of stored rows back to 16 bits, and the copy of blocks of a
// cache held in one pool.
//
// Write and read give a row of K or V D/8 lanes of 8 dims (one code word) each:
// 16-byte accesses of the 16-bit rows, and a warp holds the K and V rows of one
// (token, KV head) at D = 128 (of two at 64; one of the two rows at 256). The 64
// dims of a group sit in 8 lanes. 12301 tokens of 8 heads (64 MB each way): the write
// 20.4 us, the read-back 15.3, one after the other on the same rows 31.0; 9.5 each at the
// copy rate. No unit is full (ncu): issue slots 71 and 73 % of the cycles in which an SM
// holds warps and 56 and 51 % of all, the ALU pipe 45 and 44, DRAM 29 and 14. Most often a
// warp could issue and another one does; behind that come fixed latencies, a busy math
// pipe and, in the read-back, its loads. The write issues 159 instructions a warp and
// token row. One lane per D/32 dims of both rows, with the IEEE division of every
// element, took 63 us for both; 16 dims a lane 32.0, and 4.7 us against 4.2 for a step
// of 64 tokens.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "device_common.cuh"
#include "int4_layout.cuh"
#include "launch.h"

namespace pkv {
namespace {

template <typename T>
__device__ __forceinline__ uint16_t round_bits(float x);  // x rounded to T, its bits
template <>
__device__ __forceinline__ uint16_t round_bits<__half>(float x) { return __half_as_ushort(__float2half_rn(x)); }
template <>
__device__ __forceinline__ uint16_t round_bits<__nv_bfloat16>(float x) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
template <typename T>
__device__ __forceinline__ float from_bits(uint16_t b);
template <>
__device__ __forceinline__ float from_bits<__half>(uint16_t b) { return __half2float(__ushort_as_half(b)); }
template <>
__device__ __forceinline__ float from_bits<__nv_bfloat16>(uint16_t b) {
  return __uint_as_float(uint32_t(b) << 16);
}

// Division of n < 2^31 by a fixed d, by the method of division by invariant integers
// (Granlund and Montgomery, 1994): (n * mul) >> (32 + shift) with mul = floor(2^(31 + l) /
// d) + 1 and l = ceil(log2 d) = shift + 1 (d = 1 by itself).
struct Divisor {
  uint32_t d, mul, shift;
  explicit Divisor(uint32_t div) : d(div), mul(0), shift(0) {
    uint32_t l = 0;
    while ((uint64_t(1) << l) < d) ++l;
    if (l == 0) return;
    mul = uint32_t((uint64_t(1) << (31 + l)) / d + 1);
    shift = l - 1;
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return d == 1 ? n : __umulhi(n, mul) >> shift; }
};

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float b, float c) { return fma2(a, make_float2(b, b), make_float2(c, c)); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Which row and word a thread has: K and V rows alternate.
struct Int4Place {
  uint32_t token, head, v;  // v: 0 K, 1 V
  int word;
  // where the word lies in a tile, as kv4_k_word and kv4_v_word say: r's row
  // plus (at ^ ((r << shift) & turn))
  uint32_t at, turn, shift;
};
template <int D>
__device__ __forceinline__ Int4Place int4_place(const Divisor& heads) {
  constexpr uint32_t LPR = D / 8;  // lanes of a row
  const uint32_t i = blockIdx.x * 256u + threadIdx.x, row = i / LPR;
  Int4Place p;
  p.word = int(i % LPR);
  p.v = row & 1u;
  p.token = heads(row >> 1);
  p.head = (row >> 1) - p.token * heads.d;
  p.at = uint32_t(p.v ? kv4_v_word<D>(0, p.word) : kv4_k_word<D>(0, p.word));
  p.turn = D == 256 ? (p.v ? 0x60u : 0x40u) : D == 128 && p.v ? 0x20u : 0u;
  p.shift = D == 256 && p.v ? 5u : 4u;
  return p;
}

// Pairs of T.
template <typename T>
struct Pair2;
template <>
struct Pair2<__half> {
  using type = __half2;
  static __device__ __forceinline__ type make(__half a, __half b) { return __halves2half2(a, b); }
};
template <>
struct Pair2<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static __device__ __forceinline__ type make(__nv_bfloat16 a, __nv_bfloat16 b) { return __halves2bfloat162(a, b); }
};
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it to 0 <= x < 2^22 rounds x to an integer, ties to even

// Eight dims of a row quantised with their group (8 neighbouring lanes): codes,
// and the group's {s, z}. Minimum and maximum are taken in T (exactly, NaN
// spreading), as one pair (min, -max) across the lanes. The quotient a / b of the
// definition is a times an approximate 1 / b, whose error (a few 2^-24 of at most
// 15) matters only next to a half, where the IEEE quotient decides; so it does
// for subnormal s, which can send x past code 15.
template <typename T>
__device__ __forceinline__ uint32_t quantize8(const uint4& u, uint32_t& pair) {
  using T2 = typename Pair2<T>::type;
  const T2* e = reinterpret_cast<const T2*>(&u);
  const T2 mn = __hmin2_nan(__hmin2_nan(e[0], e[1]), __hmin2_nan(e[2], e[3]));
  const T2 mx = __hmax2_nan(__hmax2_nan(e[0], e[1]), __hmax2_nan(e[2], e[3]));
  T2 both = Pair2<T>::make(__hmin_nan(mn.x, mn.y), __hneg(__hmax_nan(mx.x, mx.y)));
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) {
    const uint32_t other = __shfl_xor_sync(kFull, *reinterpret_cast<const uint32_t*>(&both), m);
    both = __hmin2_nan(both, *reinterpret_cast<const T2*>(&other));
  }
  const float half_z = 0.5f * float(both.x), range = -0.5f * float(both.y) - half_z;  // 0.5 max - 0.5 min
  const bool finite = fabsf(range) < INFINITY;
  const uint16_t s = round_bits<T>(__fdiv_rn(range, 7.5f));
  const uint32_t nan = round_bits<T>(NAN);
  pair = finite ? uint32_t(s) | (uint32_t(round_bits<T>(float(both.x))) << 16) : nan | (nan << 16);
  const float half_s = 0.5f * from_bits<T>(s);
  float inv;  // (approximate; subnormal half_s goes the other way below)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(half_s));
  float x[8];
  Vec8<T>::to_float(u, x);
  // Dims i and i + 4 together. r is the product d inv rounded to an integer (on
  // top of kMagic), e what the rounding left, low and high the negated codes of
  // dims 0 .. 3 and 4 .. 7 as base-16 numbers (exact in fp32).
  float2 sum = make_float2(0.f, 0.f);
  float worst = 0.f;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const float2 d = fma2(make_float2(x[i], x[i + 4]), 0.5f, -half_z);
    const float2 r = fma2(d, inv, kMagic), minus = fma2(r, -1.f, kMagic);
    const float2 e = fma2(d, make_float2(inv, inv), minus);
    sum = fma2(sum, make_float2(16.f, 16.f), minus);
    worst = max3(worst, fabsf(e.x), fabsf(e.y));
  }
  uint32_t codes = __byte_perm(__float_as_uint(8388608.f - sum.x), __float_as_uint(8388608.f - sum.y), 0x5410);
  const bool near = !(half_s >= (std::is_same<T, __half>::value ? 0x1p-14f : 0x1p-100f)) || worst > 0.49999f;
  if (near) {
    codes = 0;
    if (half_s > 0.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(0.5f * x[i], half_z), half_s)), 0.f), 15.f);
        codes |= uint32_t(c) << (4 * i);
      }
    }
  }
  return finite ? codes : 0u;
}

// Byte offset in a tile of a thread's word, for slot r in tile row `row`.
template <int D>
__device__ __forceinline__ uint32_t word_offset(const Int4Place& p, uint32_t r, uint32_t row) {
  return (p.v ? r : row) * (D / 2) + (p.at ^ ((r << p.shift) & p.turn));
}
// The tile of a valid slot.
template <int D, typename Byte>
__device__ __forceinline__ Byte* tile_of(Byte* cache, const Int4Place& p, int64_t slot, uint32_t heads) {
  return cache + p.head * uint32_t(kv4_tile_bytes(D)) + uint64_t(uint32_t(slot >> 4)) * (heads * uint32_t(kv4_tile_bytes(D)));
}

// U tokens per thread, `stride` apart, all their loads in flight together: large
// calls take 4 (12301 tokens: 31.9 us, with 1 for the write 38.1, 2 34.2, 8 40.9),
// small ones 1 (more CTAs).
template <typename T, int D, int U>
__global__ void __launch_bounds__(256)
reshape_and_cache_int4_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                              unsigned char* __restrict__ cache, const int64_t* __restrict__ slots, uint32_t tokens,
                              uint32_t stride, const Divisor heads, int64_t num_slots, unsigned int* status) {
  asm volatile("griddepcontrol.launch_dependents;");
  const Int4Place p = int4_place<D>(heads);
  const uint4* src = (p.v ? v : k) + p.head * (D / 8) + p.word;
  const uint32_t pairs_at = (16 + p.v) * D + 4 * (uint32_t(p.word) / 8);  // of the group, in row 0
  const bool lead = p.word % 8 == 0;
  int64_t slot[U];
  uint4 x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t t = p.token + u * stride;
    const bool in = p.token < stride && t < tokens;  // (whole groups of 8 lanes; the others help the shuffles)
    slot[u] = in ? __ldg(slots + t) : -1;
    x[u] = in ? __ldg(src + uint64_t(t) * (heads.d * (D / 8))) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t pair;
    const uint32_t codes = quantize8<T>(x[u], pair);
    if (uint64_t(slot[u]) >= uint64_t(num_slots)) {  // (negative ones too)
      if (slot[u] >= 0 && p.head == 0 && p.word == 0) flag(status, PKV_DEV_BAD_SLOT);
      continue;
    }
    unsigned char* tile = tile_of<D>(cache, p, slot[u], heads.d);
    const uint32_t r = uint32_t(slot[u]) % kBlock, row = uint32_t(kv4_row(int(r)));
    *reinterpret_cast<uint32_t*>(tile + word_offset<D>(p, r, row)) = codes;
    if (lead) *reinterpret_cast<uint32_t*>(tile + pairs_at + row * (D / 16)) = pair;
  }
}

template <typename T, int D, int U>
__global__ void __launch_bounds__(256)
gather_cache_int4_kernel(uint4* __restrict__ k, uint4* __restrict__ v, const unsigned char* __restrict__ cache,
                         const int64_t* __restrict__ slots, uint32_t tokens, uint32_t stride, const Divisor heads,
                         int64_t num_slots, unsigned int* status) {
  const Int4Place p = int4_place<D>(heads);
  if (p.token >= stride) return;
  uint4* dst = (p.v ? v : k) + p.head * (D / 8) + p.word;
  const uint32_t pairs_at = (16 + p.v) * D + 4 * (uint32_t(p.word) / 8);
  int64_t slot[U];
  uint32_t codes[U], pair[U];
#pragma unroll
  for (int u = 0; u < U; ++u) slot[u] = p.token + u * stride < tokens ? __ldg(slots + p.token + u * stride) : -1;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    codes[u] = pair[u] = 0u;  // zeros for slots < 0
    if (slot[u] >= num_slots) {
      if (p.head == 0 && p.word == 0) flag(status, PKV_DEV_BAD_SLOT);
    } else if (slot[u] >= 0) {
      const unsigned char* tile = tile_of<D>(cache, p, slot[u], heads.d);
      const uint32_t r = uint32_t(slot[u]) % kBlock, row = uint32_t(kv4_row(int(r)));
      codes[u] = *reinterpret_cast<const uint32_t*>(tile + word_offset<D>(p, r, row));
      pair[u] = *reinterpret_cast<const uint32_t*>(tile + pairs_at + row * (D / 16));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t t = p.token + u * stride;
    if (t >= tokens) continue;
    const float s = from_bits<T>(uint16_t(pair[u] & 0xffffu)), z = from_bits<T>(uint16_t(pair[u] >> 16));
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // codes i and i + 4 as fp16: their bits under those of 1024
      const uint32_t bits = ((codes[u] >> (4 * i)) & 0x000f000fu) | 0x64006400u;
      const float2 c = __half22float2(__hsub2(*reinterpret_cast<const __half2*>(&bits), __float2half2_rn(1024.f)));
      const float2 y = fma2(c, s, z);
      x[i] = y.x;
      x[i + 4] = y.y;
    }
    dst[uint64_t(t) * (heads.d * (D / 8))] = Vec8<T>::from_float(x);
  }
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

template <typename T, int D, int U>
cudaError_t write_or_gather_u(bool gather, void* k, void* v, void* cache, const int64_t* slots, uint32_t tokens,
                              uint32_t heads, int64_t num_slots, unsigned int* status, cudaStream_t stream) {
  const uint32_t stride = (tokens + U - 1) / U;
  const unsigned ctas = unsigned((uint64_t(stride) * heads * 2 * (D / 8) + 255) / 256);
  if (gather)
    gather_cache_int4_kernel<T, D, U><<<ctas, 256, 0, stream>>>(
        static_cast<uint4*>(k), static_cast<uint4*>(v), static_cast<const unsigned char*>(cache), slots, tokens, stride,
        Divisor(heads), num_slots, status);
  else
    reshape_and_cache_int4_kernel<T, D, U><<<ctas, 256, 0, stream>>>(
        static_cast<const uint4*>(k), static_cast<const uint4*>(v), static_cast<unsigned char*>(cache), slots, tokens,
        stride, Divisor(heads), num_slots, status);
  return cudaGetLastError();
}

// Calls of more than kFewThreads threads at one token each (two waves of full
// SMs) take 4 tokens a thread.
constexpr uint64_t kFewThreads = 2ull * 152 * 2048;

template <typename T, int D>
cudaError_t write_or_gather(bool gather, void* k, void* v, void* cache, const int64_t* slots, uint32_t tokens,
                            uint32_t heads, int64_t num_slots, unsigned int* status, cudaStream_t stream) {
  return uint64_t(tokens) * heads * 2 * (D / 8) <= kFewThreads
             ? write_or_gather_u<T, D, 1>(gather, k, v, cache, slots, tokens, heads, num_slots, status, stream)
             : write_or_gather_u<T, D, 4>(gather, k, v, cache, slots, tokens, heads, num_slots, status, stream);
}

template <typename T>
cudaError_t write_or_gather_t(bool gather, void* k, void* v, void* cache, const int64_t* slots, uint32_t tokens,
                              uint32_t heads, int head_dim, int64_t num_slots, unsigned int* status,
                              cudaStream_t stream) {
  switch (head_dim) {
    case 64: return write_or_gather<T, 64>(gather, k, v, cache, slots, tokens, heads, num_slots, status, stream);
    case 128: return write_or_gather<T, 128>(gather, k, v, cache, slots, tokens, heads, num_slots, status, stream);
    case 256: return write_or_gather<T, 256>(gather, k, v, cache, slots, tokens, heads, num_slots, status, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_cache_int4(bool gather, void* k, void* v, bool bf16, void* cache, const int64_t* slots,
                              int num_tokens, int num_kv_heads, int head_dim, int num_blocks, unsigned int* status,
                              cudaStream_t stream) {
  const int64_t num_slots = int64_t(num_blocks) * kBlock;
  const uint32_t tokens = uint32_t(num_tokens), heads = uint32_t(num_kv_heads);
  return bf16 ? write_or_gather_t<__nv_bfloat16>(gather, k, v, cache, slots, tokens, heads, head_dim, num_slots, status,
                                                 stream)
              : write_or_gather_t<__half>(gather, k, v, cache, slots, tokens, heads, head_dim, num_slots, status,
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
