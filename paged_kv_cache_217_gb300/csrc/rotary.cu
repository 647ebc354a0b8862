// The cache write that rotates by position on its way: queries and keys are turned,
// keys and values go to their slots.
//
// A pair (a, b) of elements at position p and frequency i becomes
//     (a cos - b sin, b cos + a sin),   cos, sin = cos_sin[p][i], cos_sin[p][R / 2 + i],
// in fp32 with every product and sum rounded by itself (what an elementwise program
// gives, bit for bit), rounded once to the type. Pairs lie R / 2 apart, or next to each
// other (interleaved); elements from R on pass unchanged.
//
// Bound by its bytes: each row is read once and written once, the table's row of a token by
// its CTA's threads from L1. 12301 tokens of 32 query and 8 KV heads (128 elements, bf16) take
// 59 us (5.2 TB/s of their 307 MB), 64 tokens of 40 + 40 + 40 heads 2.3 us, the launch. CTAs of
// 64, 192 or 256 threads took 75, 61 and 64 us; 2, 4 or 8 pairs of vectors a thread, which
// then share their cosines and sines, 63, 60 and 94.
#include <cuda_runtime.h>

#include <cstdint>

#include "device_common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kRotaryThreads = 128;

// A thread takes two 16-byte vectors of a head: with pairs R / 2 apart vectors i and i + R / 16
// of the rotated part, or two of the rest; interleaved any two, i and i + D / 16.
template <typename T>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t t = blockIdx.x;
  const int per_head = a.head_dim / 16, rot = a.rotary_dim / 16;
  const int item = int(blockIdx.y) * kRotaryThreads + int(threadIdx.x), head = item / per_head, i = item - head * per_head;
  const int kind = head < a.num_q_heads ? 0 : head < a.num_q_heads + a.num_kv_heads ? 1 : 2;  // query, key, value
  const int h = head - (kind == 0 ? 0 : a.num_q_heads + (kind - 1) * a.num_kv_heads);
  if (h >= a.num_kv_heads && kind) return;
  int pos = a.positions[t];
  const int64_t slot = a.slots[t];
  if (pos < 0) return;
  if (pos >= a.max_positions) {
    if (item == 0) flag(a.status, PKV_DEV_BAD_POSITION);
    pos = a.max_positions - 1;
  }
  const bool keep = slot >= 0 && slot < int64_t(a.num_blocks) * kBlock;
  if (item == 0 && slot >= 0 && !keep) flag(a.status, PKV_DEV_BAD_SLOT);
  if (kind && !keep) return;
  // the thread's vectors, and whether they are rotated
  const int va = a.interleaved || i < rot ? i : 2 * i, vb = a.interleaved ? i + per_head : i < rot ? i + rot : 2 * i + 1;
  const bool turn_a = kind < 2 && (a.interleaved ? va < 2 * rot : i < rot);
  const bool turn_b = kind < 2 && (a.interleaved ? vb < 2 * rot : i < rot);
  const T* src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                 t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + int64_t(h) * a.head_dim;
  T* dst = kind == 0 ? static_cast<T*>(a.q_out) + t * a.q_out_stride + int64_t(h) * a.head_dim
                     : static_cast<T*>(kind == 1 ? a.k_pool : a.v_pool) +
                           (((slot / kBlock) * a.num_kv_heads + h) * kBlock + slot % kBlock) * a.head_dim;
  uint4 x = reinterpret_cast<const uint4*>(src)[va], y = reinterpret_cast<const uint4*>(src)[vb];
  if (turn_a || turn_b) {
    float cs[8], sn[8];  // interleaved: four of va, four of vb
    const float* row = a.cos_sin + int64_t(pos) * a.rotary_dim;
    const int half = a.rotary_dim / 2;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int at = a.interleaved ? 4 * (k ? vb : va) : 8 * i + 4 * k;
      const bool on = a.interleaved ? (k ? turn_b : turn_a) : true;
      const float4 one = make_float4(1.f, 1.f, 1.f, 1.f), none = make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 c = on ? __ldg(reinterpret_cast<const float4*>(row + at)) : one;
      const float4 s = on ? __ldg(reinterpret_cast<const float4*>(row + half + at)) : none;
      cs[4 * k] = c.x, cs[4 * k + 1] = c.y, cs[4 * k + 2] = c.z, cs[4 * k + 3] = c.w;
      sn[4 * k] = s.x, sn[4 * k + 1] = s.y, sn[4 * k + 2] = s.z, sn[4 * k + 3] = s.w;
    }
    float f[8], g[8], u[8], w[8];
    Vec8<T>::to_float(x, f);
    Vec8<T>::to_float(y, g);
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[2 * e] = __fsub_rn(__fmul_rn(f[2 * e], cs[e]), __fmul_rn(f[2 * e + 1], sn[e]));
        u[2 * e + 1] = __fadd_rn(__fmul_rn(f[2 * e + 1], cs[e]), __fmul_rn(f[2 * e], sn[e]));
        w[2 * e] = __fsub_rn(__fmul_rn(g[2 * e], cs[4 + e]), __fmul_rn(g[2 * e + 1], sn[4 + e]));
        w[2 * e + 1] = __fadd_rn(__fmul_rn(g[2 * e + 1], cs[4 + e]), __fmul_rn(g[2 * e], sn[4 + e]));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[e] = __fsub_rn(__fmul_rn(f[e], cs[e]), __fmul_rn(g[e], sn[e]));
        w[e] = __fadd_rn(__fmul_rn(g[e], cs[e]), __fmul_rn(f[e], sn[e]));
      }
    }
    if (turn_a) x = Vec8<T>::from_float(u);
    if (turn_b) y = Vec8<T>::from_float(w);
  }
  reinterpret_cast<uint4*>(dst)[va] = x;
  reinterpret_cast<uint4*>(dst)[vb] = y;
}

template <typename T>
cudaError_t launch_t(const RotaryArgs& a, cudaStream_t stream) {
  const int items = (a.num_q_heads + 2 * a.num_kv_heads) * (a.head_dim / 16);
  rotary_kernel<T><<<dim3(unsigned(a.num_tokens), unsigned((items + kRotaryThreads - 1) / kRotaryThreads)), kRotaryThreads, 0,
                     stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_t<__nv_bfloat16>(a, stream) : launch_t<__half>(a, stream);
}

}  // namespace pkv
