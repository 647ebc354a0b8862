// The cache write that rotates by position on its way: queries and keys are turned,
// keys and values go to their slots.
//
// A pair (a, b) of elements at position p and frequency i becomes
//     (a cos - b sin, b cos + a sin),   cos, sin = cos_sin[p][i], cos_sin[p][R / 2 + i],
// in fp32 with every product and sum rounded by itself (what an elementwise program
// gives, bit for bit), rounded once to the type. Pairs lie R / 2 apart, or next to each
// other (interleaved); elements from R on pass unchanged.
//
// Bound by its bytes: each row is read once and written once.
#include <cuda_runtime.h>

#include <cstdint>

#include "device_common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kRotaryThreads = 256;

// A thread takes two 16-byte vectors of a head: with pairs R / 2 apart vectors i and i + R / 16
// of the rotated part, or two of the rest; interleaved any two, i and i + D / 16. Its heads are
// kRotaryThreads / (D / 16) apart, so that the cosines and sines stay in registers.
template <typename T>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t t = blockIdx.x;
  const int per_head = a.head_dim / 16;
  const int items = (a.num_q_heads + 2 * a.num_kv_heads) * per_head;
  const int i = threadIdx.x % per_head, rot = a.rotary_dim / 16;
  int pos = a.positions[t];
  const int64_t slot = a.slots[t];
  if (pos < 0) return;
  if (pos >= a.max_positions) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag(a.status, PKV_DEV_BAD_POSITION);
    pos = a.max_positions - 1;
  }
  if (slot >= int64_t(a.num_blocks) * kBlock && threadIdx.x == 0 && blockIdx.y == 0) flag(a.status, PKV_DEV_BAD_SLOT);
  const bool keep = slot >= 0 && slot < int64_t(a.num_blocks) * kBlock;
  // vectors of this thread, and whether they are rotated
  const int va = a.interleaved || i < rot ? i : 2 * i, vb = a.interleaved ? i + per_head : i < rot ? i + rot : 2 * i + 1;
  const bool turn_a = a.interleaved ? va < 2 * rot : i < rot, turn_b = a.interleaved ? vb < 2 * rot : i < rot;
  float cs[8], sn[8];  // interleaved: four of va, four of vb
  {
    const float* row = a.cos_sin + int64_t(pos) * a.rotary_dim;
    const int half = a.rotary_dim / 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = a.interleaved ? 4 * (h ? vb : va) : 8 * i + 4 * h;
      const bool on = a.interleaved ? (h ? turn_b : turn_a) : turn_a;
      const float4 one = make_float4(1.f, 1.f, 1.f, 1.f), none = make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 c = on ? __ldg(reinterpret_cast<const float4*>(row + at)) : one;
      const float4 s = on ? __ldg(reinterpret_cast<const float4*>(row + half + at)) : none;
      cs[4 * h] = c.x, cs[4 * h + 1] = c.y, cs[4 * h + 2] = c.z, cs[4 * h + 3] = c.w;
      sn[4 * h] = s.x, sn[4 * h + 1] = s.y, sn[4 * h + 2] = s.z, sn[4 * h + 3] = s.w;
    }
  }
  for (int item = blockIdx.y * kRotaryThreads + threadIdx.x; item < items; item += gridDim.y * kRotaryThreads) {
    const int head = item / per_head;
    const int kind = head < a.num_q_heads ? 0 : head < a.num_q_heads + a.num_kv_heads ? 1 : 2;  // query, key, value
    const int h = head - (kind == 0 ? 0 : a.num_q_heads + (kind - 1) * a.num_kv_heads);
    if (kind && !keep) continue;
    const T* src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                   t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + int64_t(h) * a.head_dim;
    T* dst;
    if (kind == 0) {
      dst = static_cast<T*>(a.q_out) + t * a.q_out_stride + int64_t(h) * a.head_dim;
    } else {
      dst = static_cast<T*>(kind == 1 ? a.k_pool : a.v_pool) +
            (((slot / kBlock) * a.num_kv_heads + h) * kBlock + slot % kBlock) * a.head_dim;
    }
    uint4 x = reinterpret_cast<const uint4*>(src)[va], y = reinterpret_cast<const uint4*>(src)[vb];
    if (kind < 2 && (turn_a || turn_b)) {
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
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, bool bf16, cudaStream_t stream) {
  const int items = (a.num_q_heads + 2 * a.num_kv_heads) * (a.head_dim / 16);
  const dim3 grid(unsigned(a.num_tokens), unsigned((items + kRotaryThreads - 1) / kRotaryThreads));
  if (bf16) rotary_kernel<__nv_bfloat16><<<grid, kRotaryThreads, 0, stream>>>(a);
  else rotary_kernel<__half><<<grid, kRotaryThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
