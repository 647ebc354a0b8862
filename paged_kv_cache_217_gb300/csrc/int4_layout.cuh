// The 4-bit KV cache: numbers and tile layout.
//
// Every stored row (block, KV head, slot) of K and of V is cut into groups of
// 64 head dims. A group of a 16-bit type T keeps 4-bit codes c and a pair
// {s, z} of T with x ~= z + c * s:
//     z = min x,  s = round_T((0.5 max x - 0.5 z) / 7.5),
//     c = clamp(rint((0.5 x - 0.5 z) / (0.5 s)), 0, 15)   (c = 0 where s = 0),
// all in IEEE fp32; the halves keep the widest bf16 ranges inside fp32. z is
// one of the inputs, so it is exact, and c is taken against the rounded s, so
// the rounding of s to T widens the error of an element only beyond code 15. It is
// off by at most half a step: a relative 2^-8 for bf16 and 2^-11 for fp16, 2^-134 and
// 2^-25 where s is subnormal. So |x - (z + c s)| <= s / 2 for x <= z + 15 s, and the
// largest x passes z + 15 s by at most 15 s 2^-8 (15 s 2^-11; 15 2^-134, 15 2^-25). A
// group that holds an infinity or NaN stores NaN in both, so everything read from it
// is NaN.
//
// A tile is the 16 slots of one (block, KV head): 18 * D contiguous bytes,
//     K codes 8 D | V codes 8 D | K pairs D | V pairs D,
// so that one untiled bulk copy brings a whole tile (its address and size are
// multiples of 128). Codes are kept as 32-bit words of 8 head dims (dim
// 8 w + j in bits 4 j of word w). Rows and words are placed where the decode
// kernel's lanes read them, with no bank conflict and no shuffle:
//  * K: slot r is tile row kv4_row(r) (the order in which the tensor-core
//    fragment takes tokens), and lane t = (w % 8) / 2 of a quad reads its D/32
//    words of a row at once;
//  * V: slot r is row r; lane g = w % 8 reads its D/64 words at once, turned
//    by the row so that 4 rows 64 bytes or more apart fall into other banks;
//  * pairs: row kv4_row(r), group order, {s, z}.
#pragma once

#include <cstdint>

namespace pkv {

constexpr int kInt4Group = 64;  // head dims that share one {s, z}

__host__ __device__ constexpr int kv4_tile_bytes(int D) { return 18 * D; }

// Tile row of slot r: the token that row 2 t + b + 8 h of an MMA fragment
// stands for is 8 h + 4 b + t (t < 4), see decode_int4.cuh.
__host__ __device__ constexpr int kv4_row(int r) { return 8 * (r >> 3) + 2 * (r & 3) + ((r >> 2) & 1); }

// Byte offset in the tile of word w (head dims 8 w .. 8 w + 7) of slot r.
template <int D>
__host__ __device__ constexpr int kv4_k_word(int r, int w) {
  const int row = kv4_row(r), t = (w % 8) / 2, i = 2 * (w / 8) + w % 2;
  if (D == 256) return row * (D / 2) + 16 * ((4 * (i / 4) + t) ^ (4 * (row & 1))) + 4 * (i % 4);
  return row * (D / 2) + (D / 8) * t + 4 * i;
}

template <int D>
__host__ __device__ constexpr int kv4_v_turn(int r) {
  return D == 64 ? 0 : D == 128 ? 4 * ((r >> 1) & 1) : 2 * (r & 3);
}

template <int D>
__host__ __device__ constexpr int kv4_v_word(int r, int w) {
  return 8 * D + r * (D / 2) + (D / 16) * ((w % 8) ^ kv4_v_turn<D>(r)) + 4 * (w / 8);
}

// Byte offset of the {s, z} pair of group g of slot r (a pair is 4 bytes).
template <int D>
__host__ __device__ constexpr int kv4_k_pair(int r, int g) {
  return 16 * D + kv4_row(r) * (D / 16) + 4 * g;
}
template <int D>
__host__ __device__ constexpr int kv4_v_pair(int r, int g) {
  return 17 * D + kv4_row(r) * (D / 16) + 4 * g;
}

}  // namespace pkv
