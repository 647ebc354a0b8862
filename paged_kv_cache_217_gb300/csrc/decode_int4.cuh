// PagedAttention decode over the 4-bit KV cache on the tensor cores (sm_103a).
//
// Attention over K = z + c s and V = z + c s with one {s, z} per row and 64
// head dims (int4_layout.cuh). With q the query, per group g of 64 dims
//     q . K_t  = sum_g ( s_tg sum_d q_d c_td + z_tg sum_d q_d )
//     (p V)_d  = sum_t (p_t s_tg) c_td + sum_t p_t z_tg,      d in g,
// so the codes enter the products as they are and the pairs touch only scores
// and weights: no element is dequantised.
//
// Two 16-token tiles a step, as mma.sync m16n8k16 with fp16 inputs and fp32
// accumulators; the 8 columns of N belong to the KV head's query heads:
//  * S^T = C_K Q^T: tokens on M. A quad's lane t holds words 8 g + 2 t, + 1 of
//    its two token rows (one shared load a row). Codes become fp16 by masking
//    alone: a nibble in bits 0-3 of a half is the subnormal c 2^-24, and the
//    byte c0 + 16 c1 above and including it is exact too (a half's low 11 bits
//    are linear), both without loss in the tensor cores' products.
//    Up to 4 heads take two columns each: with A = (c0, c0 + 16 c1), column a
//    has (q0, q1 / 16) and column b (q1 / 16, 0), and a - b = q0 c0 + q1 c1: 4
//    integer instructions convert 8 codes. 5 to 8 heads, a column each, take c0
//    and c1 16 by a mask each: 5 instructions. The query is scaled by a power of
//    two per head that brings max |q| to [2^13, 2^14): bf16 and fp16 queries are
//    exact (elements below 2^-24 of the largest lose bits).
//    (e4m3 holds a nibble in a byte exactly, c 2^-9, in 3 instructions per 8
//    codes; but mma.sync on e4m3 cost 110 instructions a tile more here, as many
//    as it takes to convert to fp16.)
//    The fp32 sums of each group are then multiplied by s and joined by
//    z * sum q.
//  * O^T += C_V^T P~: head dims on M, tokens on K, fp16. V words of tokens t
//    and t + 4 (t + 8 and t + 12) are merged by halves and masked: 10
//    instructions for 16 codes (nibble_sums).
//    P~ = p s 2^e rounded to fp16 once, 2^e a power of two per warp and 64 dims that
//    keeps P~ below 2^15; the score fragment becomes the weight operand through movmatrix.
//    The offsets' part sum p z is kept in fp32 per (head, group). With fp16 values
//    7.5 times what the rounding of P~ left joins it: the products' error is then
//    2^-11 relative of p s (c - 7.5), which is as large as the values, not of p s
//    c, several times them (z is as large with the other sign). Outputs of 100
//    tokens are 0.00025 (relative, rms) from a 64-bit computation, 0.00048 without;
//    rounding them to fp16 alone gives 0.00021. Rounding to bf16 gives 0.0016, so
//    there the step is left out (it costs 2 %, 59.0 us against 57.9).
//    An element far below its 64 dims' largest scale s_max has an absolute error too: P~
//    below 2^-14 is subnormal in fp16, p s off by up to 2^-31 s_max a token.
//  * The running maximum is only a reference: it moves when a score exceeds it
//    by more than 8 (weights up to 2^8; one vote a step), so most steps need no
//    cross-lane maximum and no rescaling. Sums and the accumulator are fp32.
// One bulk copy (18 D bytes, contiguous) brings a tile; each warp runs its own
// ring of stages of two tiles.
//
// Work: the batch's tile pairs, by sequence, KV head and position, are one list,
// cut into equal ranges for the CTAs and their warps; a warp streams its range
// without a pause, its ring filled across items, so that a short sequence costs
// no start-up of its own. An item (sequence, KV head) inside one warp's range is
// written from registers; the pieces of one that spans warps meet in shared
// memory, of one that spans CTAs in the workspace (int4_merge_kernel). Small
// batches instead give each item a CTA of its own, without that second kernel.
// One CTA per item for all batches started up for 3.5 us an item: 74.4 us for 40
// heads and 64 sequences against 57.7 (58.9 now, 5.1 of the 6.8 TB/s that a copy
// reaches), where 256 sequences of 150 tokens x 8 KV heads took 22.8 against 22.3 (22.9
// now; the powers of two per 64 dims and the lifted sums are the difference): there
// the list (2 us), the block ids (1.4), the first copies (1) and the joins (4)
// stand around 7 us of streaming.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "decode.cuh"
#include "device_common.cuh"
#include "even_split.cuh"
#include "int4_layout.cuh"
#include "launch.h"

namespace pkv {

template <int D, int H, int NW, int STAGES>
struct I4Cfg {
  static constexpr int TILE_BYTES = kv4_tile_bytes(D);
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
  static constexpr int PIECE_FLOATS = H * (D + 2);  // means[H][D], m[H], l[H] of a piece
  static constexpr size_t RING_BYTES = size_t(NW) * STAGES * STAGE_BYTES;
  static constexpr size_t PIECE_BYTES = size_t(NW) * PIECE_FLOATS * sizeof(float);
  static constexpr size_t BAR_BYTES = size_t(NW) * STAGES * 8;
  static constexpr size_t SMEM_BYTES = RING_BYTES + PIECE_BYTES + BAR_BYTES + NW * 32 * 12 + NW * 64 + 64;
  static_assert(PIECE_FLOATS * 4 <= STAGES * STAGE_BYTES, "a piece fits a warp's ring");
  static_assert(PIECE_FLOATS % 4 == 0, "pieces are 16-byte aligned");
};

// Warps per CTA, and CTAs that an SM holds. Measured on GB300 at head_dim 128:
// 2 x 6 warps (168 registers) 61.2 us, 2 x 8 (128, some spilled) 65.1 on the
// 40-head layer, 115.8 against 118.9 on 96 heads x 3 long sequences; at 256 one
// CTA of 8 (255 registers) 60.4 us against 67.8 with 6 (all before the joins were
// shortened, which took 2 to 3 us off each). A prefetch of later tiles
// into L2 made all of them 5-18 % slower.
template <int D>
constexpr int i4_warps() { return D == 256 ? 8 : 6; }
template <int D>
constexpr int i4_ctas_per_sm() { return D == 256 ? 1 : 2; }
constexpr int kInt4MaxCtas = 2 * 152;  // one wave of a GB300

// Scores past the reference by more than this move it.
constexpr float kInt4Lazy = 8.f;

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t lds_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// N 32-bit words from shared memory in one load.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "what one load brings");
  if constexpr (N == 1) {
    w[0] = lds_u32(addr);
  } else if constexpr (N == 2) {
    const uint2 v = lds64(addr);
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = lds128(addr);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}

// The {s, z} of a pair word.
template <typename T>
__device__ __forceinline__ float2 pair_of(uint32_t u);
template <>
__device__ __forceinline__ float2 pair_of<__nv_bfloat16>(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 pair_of<__half>(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// A word's halves (nibbles 0..3 of each) as fp16 pairs in units of 2^-24: n0, n0
// + 16 n1, n2, n2 + 16 n3. The upper nibbles are never taken alone: the products
// of n0 + 16 n1 less those of n0 are 16 times theirs, which is sorted out where
// the products are read.
__device__ __forceinline__ void nibble_sums(uint32_t w, uint32_t (&p)[4]) {
  p[0] = w & 0x000f000fu;
  p[1] = w & 0x00ff00ffu;
  p[3] = __byte_perm(w, 0, 0x4341);  // (w >> 8) & 0x00ff00ff
  p[2] = p[3] & 0x000f000fu;
}

// A word's eight nibbles as fp16 pairs: (0, 4) and (2, 6) times 2^-24, (1, 5)
// and (3, 7) times 2^-20.
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t (&p)[4]) {
  p[0] = w & 0x000f000fu;
  p[1] = w & 0x00f000f0u;
  w >>= 8;
  p[2] = w & 0x000f000fu;
  p[3] = w & 0x00f000f0u;
}

// d = a b + c. A plain function of its operands (not volatile), so that the
// compiler may interleave the chains of a step.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Layout of the query heads over a quad's lanes. H: heads the kernel takes (4 or
// 8, the group padded up). PER_LANE heads whose scores a lane keeps, the head of
// its c-th one.
template <int H>
struct I4Heads {
  static_assert(H == 4 || H == 8, "4 heads of two columns, or 8 heads");
  static constexpr int PER_LANE = H / 4;
  static __device__ __forceinline__ int head(int t, int c) { return H == 4 ? t : 2 * t + c; }
};

// The query operand of one lane (column gr of N), and the factors of the heads
// whose scores it keeps.
template <int D, int H>
struct I4Query {
  uint32_t b[D / 16][2];                            // k-step 2 (2 g + i) + j: word 8 g + 2 t + i
  float sum[D / kInt4Group][I4Heads<H>::PER_LANE];  // sum of the scaled query over a group, times 2^-24
  float mul[I4Heads<H>::PER_LANE];                  // scale log2(e) / the power of two (2^24 is applied apart)
};

// The 16-bit query elements of a lane: dims 64 g + 16 t .. + 15 of its column's
// head (words 8 g + 2 t, + 1).
template <int D>
struct I4Raw {
  uint4 u[D / kInt4Group][2];
};
template <typename T, int D, int H>
__device__ __forceinline__ void i4_load_query(const T* q0, int group, int lane, I4Raw<D>& raw) {
  const int t = lane & 3, head = (lane >> 2) * H / 8;
#pragma unroll
  for (int g = 0; g < D / kInt4Group; ++g) {
    raw.u[g][0] = raw.u[g][1] = make_uint4(0, 0, 0, 0);
    if (head < group) {
      const uint4* src = reinterpret_cast<const uint4*>(q0 + size_t(head) * D + 64 * g + 16 * t);
      raw.u[g][0] = *src;
      raw.u[g][1] = src[1];
    }
  }
}

template <typename T, int D, int H>
__device__ __forceinline__ void i4_query(const I4Raw<D>& raw, int lane, float scale_log2, I4Query<D, H>& q) {
  using HL = I4Heads<H>;
  constexpr int GROUPS = D / kInt4Group;
  const int t = lane & 3;
  float m = 0.f;
#pragma unroll
  for (int g = 0; g < GROUPS; ++g)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x[8];
      Vec8<T>::to_float(raw.u[g][i], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
    }
  m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
  m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
  // m < 2^E (E from m's exponent field, clamped for tiny or zero q): times 2^(14 - E)
  const int E = max(int((__float_as_uint(m) >> 23) & 0xffu) - 126, -100);
  const float up = __uint_as_float(uint32_t(127 + 14 - E) << 23);
  const float mul = scale_log2 * __uint_as_float(uint32_t(127 - 14 + E) << 23);
#pragma unroll
  for (int c = 0; c < HL::PER_LANE; ++c) q.mul[c] = __shfl_sync(kFull, mul, 4 * (HL::head(t, c) * 8 / H));
  const bool col_b = H == 4 && (lane & 4);
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x[8];
      Vec8<T>::to_float(raw.u[g][i], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= up;
        sum += x[e];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const __half2 even = __floats2half2_rn(x[2 * j], x[2 * j + 4]);
        const __half2 odd = __floats2half2_rn(x[2 * j + 1] * 0.0625f, x[2 * j + 5] * 0.0625f);
        const uint32_t e = *reinterpret_cast<const uint32_t*>(&even), o = *reinterpret_cast<const uint32_t*>(&odd);
        q.b[2 * (2 * g + i) + j][0] = col_b ? o : e;
        q.b[2 * (2 * g + i) + j][1] = col_b ? 0u : o;
      }
    }
    sum += __shfl_xor_sync(kFull, sum, 1);
    sum += __shfl_xor_sync(kFull, sum, 2);
    sum *= 0x1p-24f;
#pragma unroll
    for (int c = 0; c < HL::PER_LANE; ++c) q.sum[g][c] = __shfl_sync(kFull, sum, 4 * (HL::head(t, c) * 8 / H));
  }
}

// Running state of a warp. The accumulator's columns 2t, 2t + 1 are this lane's
// heads (H = 8), or both its one head.
template <int D, int H>
struct I4State {
  static constexpr int PL = I4Heads<H>::PER_LANE;
  float o[D / 16][4];            // O^T fragments in units of 2^-24 / vmul; odd ones hold even + 16 * odd nibbles
  float z[D / kInt4Group][PL];   // this lane's part of sum p z, times 2^-40 in the groups of `lifted`
  float m[PL], l[PL];            // reference maximum (log2 domain), this lane's part of sum p
  float vmul[D / kInt4Group];    // per group: P~ = p s vmul, vmul = 2^(7 - E) for s below 2^E
  uint32_t lifted;               // bit g: see kInt4BigZ
};

// 2^e / x of a power of two x, all normal numbers.
__device__ __forceinline__ float pow2_over(int e, float x) {
  return __uint_as_float((uint32_t(254 + e) << 23) - __float_as_uint(x));
}
// a / b of powers of two; 0 where that is below 2^-126. (Exponents only: the quotient next to 2^-126 sends a
// division through its slow path, 2.5 us of 59 over 64 sequences x 40 heads.)
__device__ __forceinline__ float pow2_ratio(float a, float b) {
  return __uint_as_float(uint32_t(max(127 + int(__float_as_uint(a) >> 23) - int(__float_as_uint(b) >> 23), 0)) << 23);
}

// bf16 values reach 2^128, where the unnormalised sums p v, p up to 2^8, would pass
// fp32: from an offset of kInt4BigZ or a scale of kInt4BigS on, a group's sums are
// kept 2^-40 times as large (2^8 2^27 tokens 2^128 2^-40 fits). What leaves a warp --
// pieces of an item too -- is divided by the sum of the weights, so no larger than the
// values.
constexpr float kInt4BigZ = 0x1p80f, kInt4BigS = 0x1p76f;

// The scores (log2 domain) of tile rows gr (x[0]) and gr + 8 (x[1]).
template <typename T, int D, int H>
__device__ __forceinline__ void i4_scores(uint32_t tile, const I4Query<D, H>& q, float (&x)[2][I4Heads<H>::PER_LANE],
                                          int lane) {
  constexpr int GROUPS = D / kInt4Group, PL = I4Heads<H>::PER_LANE;
  const int t = lane & 3, gr = lane >> 2;
  uint32_t kp[2][GROUPS];
  lds_words<GROUPS>(tile + 16 * D + gr * (D / 16), kp[0]);
  lds_words<GROUPS>(tile + 16 * D + (gr + 8) * (D / 16), kp[1]);
  constexpr int PER = D == 64 ? 2 : 4;  // words a shared load brings
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int c = 0; c < PL; ++c) x[r][c] = 0.f;
#pragma unroll
  for (int c = 0; c < D / 32 / PER; ++c) {
    uint32_t w0[PER], w1[PER];
    const int at = D == 256 ? 16 * ((4 * c + t) ^ (4 * (gr & 1))) : (D / 8) * t;
    lds_words<PER>(tile + gr * (D / 2) + at, w0);
    lds_words<PER>(tile + (gr + 8) * (D / 2) + at, w1);
#pragma unroll
    for (int h = 0; h < PER / 2; ++h) {
      const int g = c * (PER / 2) + h;
      float s[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t a[4], b[4];
        if constexpr (H == 4) {
          nibble_sums(w0[2 * h + i], a);
          nibble_sums(w1[2 * h + i], b);
        } else {
          nibbles(w0[2 * h + i], a);
          nibbles(w1[2 * h + i], b);
        }
        const uint32_t* b0 = q.b[2 * (2 * g + i)];
        const uint32_t* b1 = q.b[2 * (2 * g + i) + 1];
        if (i == 0) mma_f16(s, a[0], b[0], a[1], b[1], b0[0], b0[1], 0.f, 0.f, 0.f, 0.f);
        else mma_f16(s, a[0], b[0], a[1], b[1], b0[0], b0[1], s[0], s[1], s[2], s[3]);
        mma_f16(s, a[2], b[2], a[3], b[3], b1[0], b1[1], s[0], s[1], s[2], s[3]);
      }
      const float2 k0 = pair_of<T>(kp[0][g]), k1 = pair_of<T>(kp[1][g]);
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        const float y0 = H == 4 ? s[0] - s[1] : s[e], y1 = H == 4 ? s[2] - s[3] : s[2 + e];
        x[0][e] = fmaf(y0, k0.x, fmaf(k0.y, q.sum[g][e], x[0][e]));
        x[1][e] = fmaf(y1, k1.x, fmaf(k1.y, q.sum[g][e], x[1][e]));
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int e = 0; e < PL; ++e) x[r][e] = x[r][e] * q.mul[e] * 0x1p24f;
}

// Two tiles (32 tokens from a multiple of 16); with MASK only tokens [lo, rows)
// of the 32 count, whatever the rest of the stage holds.
template <typename T, int D, int H, bool MASK>
__device__ __forceinline__ void i4_step(uint32_t stage, int lo, int rows, const I4Query<D, H>& q, I4State<D, H>& st,
                                        int lane) {
  constexpr int GROUPS = D / kInt4Group, PL = I4Heads<H>::PER_LANE, TILE = kv4_tile_bytes(D);
  const int t = lane & 3, gr = lane >> 2;
  float x[4][PL];  // rows gr, gr + 8 of the first tile, then of the second
  float2 v[4][GROUPS];
  constexpr bool WIDE = !std::is_same<T, __half>::value;  // values that sums of p v can pass fp32 with
  float smax[GROUPS] = {}, zmax = 0.f;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const uint32_t tile = stage + n * TILE;
    float y[2][PL];
    i4_scores<T, D, H>(tile, q, y, lane);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t vp[GROUPS];
      lds_words<GROUPS>(tile + 17 * D + (gr + 8 * r) * (D / 16), vp);
      const int tok = 16 * n + 8 * r + 4 * (gr & 1) + (gr >> 1);  // the token of tile row gr + 8 r
      const bool on = !MASK || (tok >= lo && tok < rows);
#pragma unroll
      for (int e = 0; e < PL; ++e) x[2 * n + r][e] = on ? y[r][e] : -INFINITY;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        v[2 * n + r][g] = on ? pair_of<T>(vp[g]) : make_float2(0.f, 0.f);
        smax[g] = fmaxf(smax[g], v[2 * n + r][g].x);
        if (WIDE) zmax = fmaxf(zmax, fabsf(v[2 * n + r][g].y));
      }
    }
  }
  float mx[PL];
  bool move = WIDE && zmax >= kInt4BigZ && st.lifted != (1u << GROUPS) - 1u;
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    move |= smax[g] >= pow2_over(7, st.vmul[g]);
  }
#pragma unroll
  for (int e = 0; e < PL; ++e) {
    mx[e] = fmaxf(fmaxf(x[0][e], x[1][e]), fmaxf(x[2][e], x[3][e]));
    move |= mx[e] > st.m[e] + kInt4Lazy;
  }
  if (__any_sync(kFull, move)) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
#pragma unroll
      for (int e = 0; e < PL; ++e) mx[e] = fmaxf(mx[e], __shfl_xor_sync(kFull, mx[e], off));
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) smax[g] = fmaxf(smax[g], __shfl_xor_sync(kFull, smax[g], off));
    }
    float al[PL];
#pragma unroll
    for (int e = 0; e < PL; ++e) {
      mx[e] = fmaxf(mx[e], st.m[e]);
      // a head without a score yet has nothing to rescale
      al[e] = st.m[e] == -INFINITY ? 0.f : fast_exp2(st.m[e] - mx[e]);
      st.m[e] = mx[e];
      st.l[e] *= al[e];
    }
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      float ratio = 1.f;
      if (smax[g] >= pow2_over(7, st.vmul[g])) {  // smax in [2^(E-1), 2^E)
        const int E = min(max(int((__float_as_uint(smax[g]) >> 23) & 0xffu) - 126, -119), 126);
        const float mul = __uint_as_float(uint32_t(127 + 7 - E) << 23);
        ratio = pow2_ratio(mul, st.vmul[g]);  // (0: what is there is nothing to the new scale)
        st.vmul[g] = mul;
      }
      float zr = 1.f;
      if (WIDE) {
        float z = smax[g] >= kInt4BigS ? kInt4BigZ : 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) z = fmaxf(z, fabsf(v[r][g].y));
        const bool big = __any_sync(kFull, z >= kInt4BigZ);
        if (big && !(st.lifted >> g & 1u)) {
          st.lifted |= 1u << g;
          zr = 0x1p-40f;
        }
      }
      const float r0 = al[0] * ratio, r1 = al[PL - 1] * ratio;
#pragma unroll
      for (int e = 0; e < PL; ++e) st.z[g][e] *= al[e] * zr;
#pragma unroll
      for (int i = 4 * g; i < 4 * g + 4; ++i) {
        st.o[i][0] *= r0;
        st.o[i][1] *= r1;
        st.o[i][2] *= r0;
        st.o[i][3] *= r1;
      }
    }
  }
#pragma unroll
  for (int g = 0; g < GROUPS; ++g)
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r][g].x *= st.vmul[g];
  if (WIDE && st.lifted != 0u) {
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const float zmul = st.lifted >> g & 1u ? 0x1p-40f : 1.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r][g].y *= zmul;
    }
  }
  float p[4][PL];
#pragma unroll
  for (int e = 0; e < PL; ++e) {
    // (nothing but -inf scores so far leaves the reference at -inf)
    const float ref = st.m[e] == -INFINITY ? 0.f : st.m[e];
#pragma unroll
    for (int r = 0; r < 4; ++r) p[r][e] = fast_exp2(x[r][e] - ref);
    st.l[e] += (p[0][e] + p[1][e]) + (p[2][e] + p[3][e]);
#pragma unroll
    for (int g = 0; g < GROUPS; ++g)
#pragma unroll
      for (int r = 0; r < 4; ++r) st.z[g][e] = fmaf(p[r][e], v[r][g].y, st.z[g][e]);
  }

  // O^T += C_V^T P~: K slot 2t + b + 8h of a tile is token 8h + 4b + t.
  const int turn = D == 64 ? 0 : D == 128 ? 4 * (t >> 1) : 2 * t;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const uint32_t vt = stage + n * TILE + 8 * D + t * (D / 2) + (D / 16) * (gr ^ turn);
    uint32_t wa[GROUPS], wb[GROUPS], wc[GROUPS], wd[GROUPS];
    lds_words<GROUPS>(vt, wa);
    lds_words<GROUPS>(vt + 4 * (D / 2), wb);
    lds_words<GROUPS>(vt + 8 * (D / 2), wc);
    lds_words<GROUPS>(vt + 12 * (D / 2), wd);
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      uint32_t pb[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float s = v[2 * n + r][g].x;
        const float x0 = p[2 * n + r][0] * s, x1 = p[2 * n + r][PL - 1] * s;
        const __half2 h = __floats2half2_rn(x0, x1);
        if constexpr (std::is_same<T, __half>::value) {
          // what the rounding left goes with the offsets, as if every code were 7.5
          const float2 back = __half22float2(h);
          const float left = 7.5f * pow2_over(0, st.vmul[g]);
          st.z[g][0] = fmaf(x0 - back.x, left, st.z[g][0]);
          if (PL == 2) st.z[g][PL - 1] = fmaf(x1 - back.y, left, st.z[g][PL - 1]);
        }
        pb[r] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // nibbles 0..3, then 4..7
        uint32_t ab[4], cd[4];
        nibble_sums(__byte_perm(wa[g], wb[g], h ? 0x7632 : 0x5410), ab);
        nibble_sums(__byte_perm(wc[g], wd[g], h ? 0x7632 : 0x5410), cd);
        float(&o0)[4] = st.o[4 * g + 2 * h];
        float(&o1)[4] = st.o[4 * g + 2 * h + 1];
        mma_f16(o0, ab[0], ab[2], cd[0], cd[2], pb[0], pb[1], o0[0], o0[1], o0[2], o0[3]);
        mma_f16(o1, ab[1], ab[3], cd[1], cd[3], pb[0], pb[1], o1[0], o1[1], o1[2], o1[3]);
      }
    }
  }
}

// Sums over a quad's rows what the warp keeps by lane; lifted groups' o takes 2^40 of
// its unit.
template <int D, int H>
__device__ __forceinline__ void i4_reduce(I4State<D, H>& st) {
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
#pragma unroll
    for (int c = 0; c < I4Heads<H>::PER_LANE; ++c) {
      st.l[c] += __shfl_xor_sync(kFull, st.l[c], off);
#pragma unroll
      for (int g = 0; g < D / kInt4Group; ++g) st.z[g][c] += __shfl_xor_sync(kFull, st.z[g][c], off);
    }
  }
  if (st.lifted) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[i][e] *= st.lifted >> (i / 4) & 1u ? 0x1p40f : 1.f;
  }
}

// The reduced state's values of column c times inv, which is at most 1 (a weight next
// to the reference is 1 or more): calls f(dim, four values of dims dim .. dim + 3). Row
// gr of fragment 4 g + 2 h is dim 64 g + 8 gr + 4 h, of the next one the dim after it,
// row gr + 8 two dims on. A unit of o is 2^24 / vmul, which alone passes fp32 for scales
// from 2^110 on; those are lifted (kInt4BigS), and i4_reduce has taken 2^40 of it.
template <int D, int H, typename F>
__device__ __forceinline__ void i4_values(const I4State<D, H>& st, int c, int gr, float inv, F f) {
#pragma unroll
  for (int i = 0; i < D / 16; i += 2) {
    const float k = inv * (st.lifted >> (i / 4) & 1u ? 0x1p40f : 1.f);
    const float z = st.z[i / 4][c] * k, even = pow2_ratio(st.lifted >> (i / 4) & 1u ? 0x1p-16f : 0x1p24f, st.vmul[i / 4]) * inv,
                odd = even * 0.0625f;
    f(64 * (i / 4) + 8 * gr + 4 * ((i / 2) & 1),
      make_float4(fmaf(st.o[i][c], even, z), fmaf(st.o[i + 1][c] - st.o[i][c], odd, z), fmaf(st.o[i][2 + c], even, z),
                  fmaf(st.o[i + 1][2 + c] - st.o[i][2 + c], odd, z)));
  }
}

// Pieces of an item hold weighted means and join with weights w_i l_i / sum w l, each
// at most 1. A piece without a weight (all scores -inf) has the mean 0.
__device__ __forceinline__ float i4_inverse(float l) { return l > 0.f ? 1.f / l : 0.f; }

// A piece of an item in shared memory: means[H][D], m[H], l[H].
template <int D, int H>
__device__ __forceinline__ void i4_publish(float* piece, I4State<D, H>& st, int lane) {
  using HL = I4Heads<H>;
  const int t = lane & 3, gr = lane >> 2;
  i4_reduce<D, H>(st);
#pragma unroll
  for (int c = 0; c < HL::PER_LANE; ++c) {
    const int head = HL::head(t, c);
    i4_values<D, H>(st, c, gr, i4_inverse(st.l[c]),
                    [&](int dim, const float4& v) { *reinterpret_cast<float4*>(piece + head * D + dim) = v; });
    if (gr == 0) {
      piece[H * D + head] = st.m[c];
      piece[H * D + H + head] = st.l[c];
    }
  }
}

// A whole item's output rows.
template <typename T, int D, int H>
__device__ __forceinline__ void i4_write(T* out, int group, I4State<D, H>& st, int lane) {
  using HL = I4Heads<H>;
  const int t = lane & 3, gr = lane >> 2;
  i4_reduce<D, H>(st);
#pragma unroll
  for (int c = 0; c < HL::PER_LANE; ++c) {
    const int head = HL::head(t, c);
    if (head >= group) continue;
    i4_values<D, H>(st, c, gr, 1.f / st.l[c], [&](int dim, const float4& v) {
      T x[4] = {T(v.x), T(v.y), T(v.z), T(v.w)};
      *reinterpret_cast<uint2*>(out + size_t(head) * D + dim) = *reinterpret_cast<const uint2*>(x);
    });
  }
}

template <int D, int H>
__device__ __forceinline__ void i4_clear(I4State<D, H>& st) {
#pragma unroll
  for (int i = 0; i < D / 16; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
#pragma unroll
  for (int e = 0; e < I4Heads<H>::PER_LANE; ++e) {
    st.m[e] = -INFINITY;
    st.l[e] = 0.f;
#pragma unroll
    for (int i = 0; i < D / kInt4Group; ++i) st.z[i][e] = 0.f;
  }
#pragma unroll
  for (int g = 0; g < D / kInt4Group; ++g) st.vmul[g] = 0x1p126f;
  st.lifted = 0u;
}

// ---- work ---------------------------------------------------------------------
// A sequence's tiles and pairs of tiles (with a sliding window those that it
// touches).
struct I4Seq {
  int L, t0, nt, np, head;  // length, first tile, tiles, pairs, rows of the first tile before the window
};
__device__ __forceinline__ int i4_len(const Int4Args& a, int s) {
  const int L = a.context_lens[s], most = a.max_blocks_per_seq * kBlock;
  return L < 0 ? 0 : L > most ? most : L;
}
__device__ __forceinline__ I4Seq i4_seq(const Int4Args& a, int L) {
  const TokenRange tr = token_range(L, a.window);
  I4Seq q;
  q.L = L;
  q.t0 = tr.aligned / kBlock;
  q.nt = (L + kBlock - 1) / kBlock - q.t0;
  q.np = (q.nt + 1) / 2;
  q.head = tr.first - tr.aligned;
  return q;
}

template <int NW>
struct I4Shared {
  long long before[NW * 32];     // per thread: where its run of sequences starts in the list
  long long scan[NW], last[NW];  // per warp: ... and the last pair of the item of its last piece
  int len[NW * 32];              // per thread: the length of its run's last sequence
  int fitem[NW], fend[NW], litem[NW];
};

constexpr int kInt4NoPiece = -1, kInt4NoWork = -2;

template <typename T, int D, int H, int NW, int STAGES>
__global__ void __launch_bounds__(NW * 32, i4_ctas_per_sm<D>()) paged_decode_int4_kernel(const Int4Args a) {
  using C = I4Cfg<D, H, NW, STAGES>;
  extern __shared__ __align__(1024) unsigned char smem[];
  I4Shared<NW>& sh = *reinterpret_cast<I4Shared<NW>*>(smem + C::RING_BYTES + C::PIECE_BYTES + C::BAR_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int Hkv = a.num_kv_heads;
  unsigned char* ring = smem + size_t(warp) * STAGES * C::STAGE_BYTES;
  float* const first_piece = reinterpret_cast<float*>(smem + C::RING_BYTES) + warp * C::PIECE_FLOATS;
  const uint32_t ring_s = smem_addr(ring);
  const uint32_t bar_s = smem_addr(smem + C::RING_BYTES + C::PIECE_BYTES) + warp * STAGES * 8;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < STAGES; ++i) mbar_init(bar_s + 8 * i, 1);
    mbar_init_fence();
  }
  __syncwarp();  // a warp's other lanes use its barriers; with an item a CTA nothing else orders that
  asm volatile("griddepcontrol.launch_dependents;");
  // (what follows reads by plain loads: read-only ones are for what no running
  // kernel writes, and the last kernel may have run until now)
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // This CTA's range [cb, ce) of the list of total pairs, this warp's [wb, we),
  // and the sequence in which the latter starts.
  long long cb, ce, total, base;
  EvenSplit split(0, 1);
  int s, L;
  auto warp_begin = [&](int w) { return cb + (ce - cb) * w / NW; };
  if (a.item_ctas) {  // one item: the list is its own
    s = int(blockIdx.x) / Hkv;
    const int raw = a.context_lens[s], g = int(blockIdx.x) - s * Hkv;
    L = i4_len(a, s);
    if (raw != L && g == 0 && tid == 0) flag(a.status, PKV_DEV_BAD_CONTEXT_LEN);
    const int np = i4_seq(a, L).np;
    if (np == 0) {
      uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + (size_t(s) * a.num_q_heads + g * a.group) * D);
      for (int i = tid; i < a.group * D / 8; i += NW * 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
      return;
    }
    base = -(long long)g * np;
    cb = 0;
    ce = total = np;
  } else {
    // The tables' way into L2 begins while the lengths are read (tables of up to
    // 1 MB: a line a thread).
    const size_t line = size_t(blockIdx.x * (NW * 32u) + tid) * 32, ids = size_t(a.num_seqs) * a.max_blocks_per_seq;
    if (ids <= (1u << 18) && line < ids) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.block_tables + line));
    // Each thread sums a run of sequences, a scan of the sums gives every run's
    // place in the list, and each warp searches the places for its own start.
    int zero_len = int(blockIdx.x) < a.num_seqs ? i4_len(a, int(blockIdx.x)) : 1;  // (read along with the others)
    const int per = (a.num_seqs + NW * 32 - 1) / (NW * 32), most = a.max_blocks_per_seq * kBlock;
    const int run0 = min(a.num_seqs, tid * per), run1 = min(a.num_seqs, run0 + per);
    long long mine = 0;
    int run_len = 0;
    for (int i0 = run0; i0 < run1; i0 += 4) {
      int raw[4];  // (loads together)
#pragma unroll
      for (int j = 0; j < 4; ++j) raw[j] = i0 + j < run1 ? a.context_lens[i0 + j] : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i0 + j >= run1) break;
        run_len = raw[j] < 0 ? 0 : raw[j] > most ? most : raw[j];
        if (raw[j] != run_len && blockIdx.x == 0) flag(a.status, PKV_DEV_BAD_CONTEXT_LEN);
        mine += (long long)i4_seq(a, run_len).np * Hkv;
      }
    }
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) sh.scan[warp] = upto;
    __syncthreads();
    long long before = upto - mine;
    total = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      if (i < warp) before += sh.scan[i];
      total += sh.scan[i];
    }
    sh.before[tid] = before;
    sh.len[tid] = run_len;
    split = EvenSplit(total, a.ctas);
    cb = split.begin(int(blockIdx.x));
    ce = split.begin(int(blockIdx.x) + 1);
    // Sequences without tokens: zeros, spread over the CTAs.
    for (int i = int(blockIdx.x); i < a.num_seqs;) {
      if (zero_len == 0) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + size_t(i) * a.num_q_heads * D);
        for (int j = tid; j < a.num_q_heads * D / 8; j += NW * 32) o[j] = make_uint4(0u, 0u, 0u, 0u);
      }
      i += int(gridDim.x);
      if (i < a.num_seqs) zero_len = i4_len(a, i);
    }
    __syncthreads();
    // the last run that starts at or before the warp's first pair holds it (runs
    // that hold nothing start where the next one does)
    const long long x = warp_begin(warp);
    int r = -1;
#pragma unroll
    for (int i = 0; i < NW; ++i) r += __popc(__ballot_sync(kFull, sh.before[32 * i + lane] <= x));
    s = min(a.num_seqs, r * per);
    base = sh.before[r];
    L = sh.len[r];
    if (per > 1 && x < total) {
      for (;; ++s) {
        L = i4_len(a, s);
        const long long n = (long long)i4_seq(a, L).np * Hkv;
        if (base + n > x) break;
        base += n;
      }
    }
  }
  const long long wb = warp_begin(warp), we = warp_begin(warp + 1);
  int item = 0, ahead = 0;  // the item at hand; the next sequence's length
  I4Seq sq{};
  int g = 0, pr = 0;        // its KV head, the pair at hand
  int fitem = kInt4NoWork, fend = 0, litem = kInt4NoWork;
  if (wb < we) {
    fitem = litem = kInt4NoPiece;
    const int n_my = int(we - wb);
    sq = i4_seq(a, L);
    g = int((wb - base) / sq.np);
    pr = int(wb - base - (long long)g * sq.np);
    if (!a.item_ctas && s + 1 < a.num_seqs) ahead = i4_len(a, s + 1);

    I4Raw<D> raw;
    i4_load_query<T, D, H>(static_cast<const T*>(a.q) + (size_t(s) * a.num_q_heads + g * a.group) * D, a.group, lane, raw);

    // Copies: lanes 2 (k % 16), + 1 of `tiles` hold the pool tiles of the warp's
    // k-th pair (batches of 16, the next one read ahead; -1: none). Each lane
    // walks the list by itself.
    int cs = s, cfrom = int(base - wb);  // a lane's sequence and its place, from the warp's first pair
    I4Seq c = sq;
    auto load_tiles = [&](int batch) -> int {
      const int x = batch * 16 + (lane >> 1);
      if (x >= n_my) return -1;
      while (x >= cfrom + c.np * Hkv) {
        cfrom += c.np * Hkv;
        c = i4_seq(a, i4_len(a, ++cs));
      }
      const int at = x - cfrom, cg = at / c.np, j = 2 * (at - cg * c.np) + (lane & 1);
      if (j >= c.nt) return -1;
      int id = a.block_tables[size_t(cs) * a.max_blocks_per_seq + c.t0 + j];
      if (id < 0 || id >= a.num_blocks) {
        flag(a.status, PKV_DEV_BAD_BLOCK_ID);
        id = 0;
      }
      return id * Hkv + cg;
    };
    const unsigned char* cache = static_cast<const unsigned char*>(a.cache);
    int tiles = load_tiles(0), tiles_next = n_my > 16 ? load_tiles(1) : -1, batch = 0;
    auto issue = [&](int k) {  // warp-uniform; k increases by one per call
      if ((k >> 4) != batch) {
        tiles = tiles_next;
        ++batch;
        tiles_next = (batch + 1) * 16 < n_my ? load_tiles(batch + 1) : -1;
      }
      // the two lanes that hold the pair's tiles copy them
      const int i1 = __shfl_sync(kFull, tiles, 2 * (k & 15) + 1);
      if ((lane >> 1) == (k & 15)) {
        const int st = k % STAGES, b = lane & 1;
        const uint32_t bar = bar_s + 8 * st;
        if (b == 0) mbar_arrive_expect_tx(bar, i1 >= 0 ? C::STAGE_BYTES : C::TILE_BYTES);
        if (tiles >= 0)
          bulk_g2s(ring_s + st * C::STAGE_BYTES + b * C::TILE_BYTES, cache + size_t(tiles) * C::TILE_BYTES,
                   C::TILE_BYTES, bar);
      }
    };
    for (int k = 0; k < STAGES && k < n_my; ++k) issue(k);

    I4State<D, H> st;
    int k = 0;
    bool ok = true;
    while (k < n_my) {
      item = s * Hkv + g;
      const size_t row = size_t(s) * a.num_q_heads + g * a.group;
      I4Query<D, H> q;
      i4_query<T, D, H>(raw, lane, a.scale_log2, q);
      i4_clear<D, H>(st);
      const bool mid = pr > 0;  // the item began in another warp's range
      const int stop = min(sq.np, pr + n_my - k);
      for (; pr < stop; ++pr, ++k) {
        const int stage = k % STAGES;
        ok = ok && __all_sync(kFull, mbar_wait_bounded(bar_s + 8 * stage, (k / STAGES) & 1));
        if (!ok) break;
        const int rows = sq.L - (sq.t0 + 2 * pr) * kBlock;
        const int lo = pr == 0 ? sq.head : 0;
        const uint32_t at = ring_s + stage * C::STAGE_BYTES;
        if (rows >= 2 * kBlock && lo == 0)
          i4_step<T, D, H, false>(at, 0, 2 * kBlock, q, st, lane);
        else
          i4_step<T, D, H, true>(at, lo, rows, q, st, lane);
        __syncwarp();
        if (k + STAGES < n_my) issue(k + STAGES);
      }
      if (!ok) {
        // a copy never completed: record it, wait (bounded) for the others in flight, stop
        if (lane == 0) flag(a.status, PKV_DEV_WAIT_TIMEOUT);
        const int last = min(n_my, k + STAGES);
        for (int kk = k; kk < last; ++kk) mbar_wait_bounded(bar_s + 8 * (kk % STAGES), (kk / STAGES) & 1);
        break;
      }
      const bool done = pr == sq.np;
      if (done && k < n_my) {  // on to the next item: its query is read while this one is written
        pr = 0;
        if (++g == Hkv) {
          g = 0;
          do {  // (sequences without tokens have no place in the list)
            base += (long long)sq.np * Hkv;
            ++s;
            sq = i4_seq(a, ahead);
            ahead = s + 1 < a.num_seqs ? i4_len(a, s + 1) : 0;
          } while (sq.np == 0);
        }
        i4_load_query<T, D, H>(static_cast<const T*>(a.q) + (size_t(s) * a.num_q_heads + g * a.group) * D, a.group, lane,
                               raw);
      }
      if (mid) {
        i4_publish<D, H>(first_piece, st, lane);
        fitem = item;
        fend = done ? 1 : 0;
      } else if (done) {
        i4_write<T, D, H>(static_cast<T*>(a.out) + row * D, a.group, st, lane);
      } else {  // the range ends inside the item: every copy has landed, the ring is free
        i4_publish<D, H>(reinterpret_cast<float*>(ring), st, lane);
        litem = item;
      }
    }
  }
  if (lane == 0) {
    sh.fitem[warp] = fitem;
    sh.fend[warp] = fend;
    sh.litem[warp] = litem;
    sh.last[warp] = base + (long long)(g + 1) * sq.np - 1;
  }
  __syncthreads();
  // The runs of pieces to join: one from each warp's last piece (run r of warp r)
  // and, run NW, the pieces of an item that began in an earlier CTA; each goes on
  // with the first pieces that belong to its item. Every warp works this out by
  // itself, and the warps take the runs' rows (32 vectors of 4 dims) in turn.
  const int fit = lane < NW ? sh.fitem[lane] : kInt4NoWork;
  const unsigned ends = __ballot_sync(kFull, lane < NW && sh.fend[lane] != 0);
  const unsigned working = __ballot_sync(kFull, fit != kInt4NoWork);
  const int early = __shfl_sync(kFull, fit, working ? __ffs(working) - 1 : 0);
  const int run_item = lane < NW ? sh.litem[lane] : lane == NW ? early : kInt4NoWork;
  unsigned runs = __ballot_sync(kFull, run_item >= 0);
  const int rows = a.group * (D / 4), chunks = (rows + 31) / 32;
  int chunk = warp;
  bool open = false;
  for (; runs; runs &= runs - 1) {
    const int r = __ffs(runs) - 1, it = __shfl_sync(kFull, run_item, r);
    const unsigned pieces = __ballot_sync(kFull, fit == it);
    const bool whole = r < NW && ((pieces & ends) != 0u || a.item_ctas);
    if (r < NW && !whole) {
      // the merge's descriptor: an item that starts here and goes on, and the CTA
      // that holds its last pair
      if (tid == 0) a.desc[blockIdx.x] = make_int2(it, split.of(sh.last[r]));
      open = true;
    }
    const int is = it / Hkv, ig = it - is * Hkv;
    T* const out = static_cast<T*>(a.out) + (size_t(is) * a.num_q_heads + ig * a.group) * D;
    const size_t row = (size_t(2) * blockIdx.x + (r < NW ? 1 : 0)) * a.group;  // of its partial result
    const unsigned char* const own = smem + size_t(min(r, NW - 1)) * STAGES * C::STAGE_BYTES;  // its first piece
    for (; chunk < chunks; chunk += NW) {
      const int e = 32 * chunk + lane, h = e / (D / 4), d = e % (D / 4) * 4;
      if (e >= rows) continue;
      float m[NW + 1], l[NW + 1], M = -INFINITY, den = 0.f;
      float4 x[NW + 1], num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w <= NW; ++w) {  // (all loads together)
        const float* p = reinterpret_cast<const float*>(w < NW ? smem + C::RING_BYTES + w * (C::PIECE_FLOATS * 4) : own);
        const bool on = w < NW ? (pieces >> w) & 1u : r < NW;
        m[w] = on ? p[H * D + h] : -INFINITY;
        l[w] = on ? p[H * D + H + h] : 0.f;
        x[w] = on ? *reinterpret_cast<const float4*>(p + h * D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        M = fmaxf(M, m[w]);
      }
      const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w <= NW; ++w) {
        l[w] *= fast_exp2(m[w] - ref);
        den += l[w];
      }
      const float inv = whole ? 1.f / den : i4_inverse(den);
#pragma unroll
      for (int w = 0; w <= NW; ++w) {
        const float wt = l[w] * inv;
        num.x = fmaf(wt, x[w].x, num.x);
        num.y = fmaf(wt, x[w].y, num.y);
        num.z = fmaf(wt, x[w].z, num.z);
        num.w = fmaf(wt, x[w].w, num.w);
      }
      if (whole) {
        T y[4] = {T(num.x), T(num.y), T(num.z), T(num.w)};
        *reinterpret_cast<uint2*>(out + size_t(h) * D + d) = *reinterpret_cast<const uint2*>(y);
      } else {
        *reinterpret_cast<float4*>(a.part_o + (row + h) * D + d) = num;
        if (d == 0) a.part_ml[row + h] = make_float2(M, den);
      }
    }
    chunk -= chunks;
  }
  if (tid == 0 && !open && !a.item_ctas) a.desc[blockIdx.x] = make_int2(-1, 0);
}

// Joins the pieces of the item that starts in CTA blockIdx.x's range and goes on
// past it, one query head per CTA here, 4 dims per thread: few pieces in one round
// of loads; many by 8 (D = 64: 16) groups of threads, every 8th piece each, the
// first of which are read while the weights of all are made.
constexpr int kInt4FewPieces = 4;
template <typename T, int D>
__global__ void __launch_bounds__(256) int4_merge_kernel(const Int4Args a) {
  constexpr int LANES = D / 4, GROUPS = 256 / LANES;
  __shared__ float weight[kInt4MaxCtas], red[8];
  __shared__ float4 other[GROUPS][LANES];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c0 = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, group = tid / LANES, d = tid % LANES * 4;
  const int2 desc = __ldcg(a.desc + c0);
  if (desc.x < 0) return;
  const int n = desc.y - c0 + 1;
  auto slot = [&](int i) { return (size_t(2) * (c0 + i) + (i == 0 ? 1 : 0)) * a.group + h; };
  auto write = [&](const float4& num) {
    const int s = desc.x / a.num_kv_heads, g = desc.x - s * a.num_kv_heads;
    T x[4] = {T(num.x), T(num.y), T(num.z), T(num.w)};
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (size_t(s) * a.num_q_heads + g * a.group + h) * D + d) =
        *reinterpret_cast<const uint2*>(x);
  };
  if (n <= kInt4FewPieces) {  // one round of loads
    if (group) return;
    float2 ml[kInt4FewPieces];
    float4 o[kInt4FewPieces], num = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, den = 0.f;
#pragma unroll
    for (int i = 0; i < kInt4FewPieces; ++i) {
      ml[i] = i < n ? __ldcg(a.part_ml + slot(i)) : make_float2(-INFINITY, 0.f);
      o[i] = i < n ? __ldcg(reinterpret_cast<const float4*>(a.part_o + slot(i) * D + d)) : num;
      M = fmaxf(M, ml[i].x);
    }
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int i = 0; i < kInt4FewPieces; ++i) {
      ml[i].y *= fast_exp2(ml[i].x - ref);
      den += ml[i].y;
    }
    const float inv = 1.f / den;
#pragma unroll
    for (int i = 0; i < kInt4FewPieces; ++i) {
      const float w = ml[i].y * inv;
      num.x = fmaf(w, o[i].x, num.x);
      num.y = fmaf(w, o[i].y, num.y);
      num.z = fmaf(w, o[i].z, num.z);
      num.w = fmaf(w, o[i].w, num.w);
    }
    write(num);
    return;
  }
  constexpr int AHEAD = 8;  // pieces read while the weights are made
  float4 early[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    const int i = group + k * GROUPS;
    early[k] = i < n ? __ldcg(reinterpret_cast<const float4*>(a.part_o + slot(i) * D + d))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float M = -INFINITY;
  for (int i = tid; i < n; i += 256) {
    weight[i] = __ldcg(&a.part_ml[slot(i)].x);
    M = fmaxf(M, weight[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
  if ((tid & 31) == 0) red[tid >> 5] = M;
  __syncthreads();
  M = red[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) M = fmaxf(M, red[i]);
  const float ref = M == -INFINITY ? 0.f : M;
  float den = 0.f;
  for (int i = tid; i < n; i += 256) {
    const float w = fast_exp2(weight[i] - ref) * __ldcg(&a.part_ml[slot(i)].y);
    weight[i] = w;
    den += w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(kFull, den, o);
  __syncthreads();
  if ((tid & 31) == 0) red[tid >> 5] = den;
  __syncthreads();
  den = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) den += red[i];
  const float inv = 1.f / den;
  float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int i, const float4& o) {
    const float w = weight[i] * inv;
    num.x = fmaf(w, o.x, num.x);
    num.y = fmaf(w, o.y, num.y);
    num.z = fmaf(w, o.z, num.z);
    num.w = fmaf(w, o.w, num.w);
  };
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (group + k * GROUPS < n) add(group + k * GROUPS, early[k]);
#pragma unroll 4
  for (int i = group + AHEAD * GROUPS; i < n; i += GROUPS)
    add(i, __ldcg(reinterpret_cast<const float4*>(a.part_o + slot(i) * D + d)));
  other[group][tid % LANES] = num;
  __syncthreads();
  if (group) return;
#pragma unroll
  for (int i = 1; i < GROUPS; ++i) {
    const float4 x = other[i][tid];
    num.x += x.x;
    num.y += x.y;
    num.z += x.z;
    num.w += x.w;
  }
  write(num);
}

}  // namespace pkv
