// PagedAttention decode over the 4-bit KV cache on the tensor cores (sm_103a).
//
// Attention over K = z + c s and V = z + c s with one {s, z} per row and 64
// head dims (int4_layout.cuh). With q the query, per group g of 64 dims
//     q . K_t  = sum_g ( s_tg sum_d q_d c_td + z_tg sum_d q_d )
//     (p V)_d  = sum_t (p_t s_tg) c_td + sum_t p_t z_tg,      d in g,
// so the codes enter the products as they are and the pairs touch only scores
// and weights: no element is dequantised.
//
// Per 16-token tile, two chains of mma.sync m16n8k16 (fp16 in, fp32 out) with
// the 8 columns of N taken by the KV head's query heads (zero past the group):
//  * S^T = C_K Q~^T: tokens on M. A quad's lane t holds words 8 g + 2 t, + 1 of
//    its two token rows (one shared load a row). A word's 8 nibbles become four
//    fp16 pairs by masking alone: nibble j (bits 0-3 of a half) is the fp16
//    subnormal c 2^-24, the one above it (bits 4-7) c 2^-20, both exact in the
//    tensor cores' products, so 5 integer instructions convert 8 codes. Q~
//    holds the query of the odd dims divided by 16 to match, and is scaled by
//    a power of two per head that brings max |q| to [2^13, 2^14): bf16 and
//    fp16 queries are exact (elements below 2^-24 of the largest lose bits).
//    The fp32 sums of each group are then multiplied by s and joined by
//    z * sum q.
//  * O^T += C_V^T P~: head dims on M, tokens on K. V words of tokens t and
//    t + 4 (t + 8 and t + 12) are merged by halves and masked the same way.
//    P~ = p s 2^e rounded to fp16 once (2^-11 relative, far below the codes'
//    own step), e a power of two per warp that keeps P~ below 2^15; the score
//    fragment becomes the weight operand through movmatrix. The offsets' part
//    sum p z is kept in fp32 per (head, group).
//  * The running maximum is only a reference: it moves when a score exceeds it
//    by more than 8 (weights up to 2^8; one vote a tile), so most tiles need no
//    cross-lane maximum and no rescaling. Sums and the accumulator are fp32.
// One bulk copy (18 D bytes, contiguous) brings a tile; each warp runs its own
// ring of stages, as in the other decode kernels.
#pragma once

#include <cuda_fp16.h>

#include "decode.cuh"
#include "decode_mma.cuh"
#include "int4_layout.cuh"

namespace pkv {

template <int D, int NW, int STAGES>
struct I4Cfg {
  static constexpr int GROUPS = D / kInt4Group;
  static constexpr int TILE_BYTES = kv4_tile_bytes(D);
  static constexpr size_t RING_BYTES = size_t(NW) * STAGES * TILE_BYTES;
  static constexpr size_t SMEM_BYTES = RING_BYTES + size_t(NW) * STAGES * 8;
};

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

// N 32-bit words from shared memory in one load (N = 1, 2, 4) or two (8).
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
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

// A word's eight nibbles as fp16 pairs: (0, 4) and (2, 6) times 2^-24, (1, 5)
// and (3, 7) times 2^-20.
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t (&p)[4]) {
  p[0] = w & 0x000f000fu;
  p[1] = w & 0x00f000f0u;
  w >>= 8;
  p[2] = w & 0x000f000fu;
  p[3] = w & 0x00f000f0u;
}

// The query operand of one lane: head gr, and the per-head factors of heads
// 2t, 2t + 1 (the columns of this lane's scores).
template <int D>
struct I4Query {
  uint32_t b[D / 16][2];        // k-step 2 (2 g + i) + j: word 8 g + 2 t + i, nibbles (2j, 2j + 4), (2j + 1, 2j + 5)
  float sum[D / kInt4Group][2]; // sum of the scaled query over a group, times 2^-24
  float mul[2];                 // scores to the log2 domain: scale log2(e) / the power of two (times 2^24, applied apart)
};

template <typename T, int D>
__device__ __forceinline__ void i4_query(const T* qrow, int lane, float scale_log2, I4Query<D>& q) {
  constexpr int GROUPS = D / kInt4Group;
  const int t = lane & 3;
  float f[GROUPS][16], m = 0.f;
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (qrow) {
      const uint4* src = reinterpret_cast<const uint4*>(qrow + 64 * g + 16 * t);
      u[0] = __ldg(src);
      u[1] = __ldg(src + 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x[8];
      Vec8<T>::to_float(u[i], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[g][8 * i + e] = x[e];
        m = fmaxf(m, fabsf(x[e]));
      }
    }
  }
  m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
  m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
  // m < 2^E (E from m's exponent field, clamped for tiny or zero q): times 2^(14 - E)
  const int E = max(int((__float_as_uint(m) >> 23) & 0xffu) - 126, -100);
  const float up = __uint_as_float(uint32_t(127 + 14 - E) << 23);
  const float mul = scale_log2 * __uint_as_float(uint32_t(127 - 14 + E) << 23);
  q.mul[0] = __shfl_sync(kFull, mul, 8 * t);
  q.mul[1] = __shfl_sync(kFull, mul, 8 * t + 4);
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* x = &f[g][8 * i];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const __half2 even = __floats2half2_rn(x[2 * j] * up, x[2 * j + 4] * up);
        const __half2 odd = __floats2half2_rn(x[2 * j + 1] * (up * 0.0625f), x[2 * j + 5] * (up * 0.0625f));
        q.b[2 * (2 * g + i) + j][0] = *reinterpret_cast<const uint32_t*>(&even);
        q.b[2 * (2 * g + i) + j][1] = *reinterpret_cast<const uint32_t*>(&odd);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += x[e] * up;
    }
    sum += __shfl_xor_sync(kFull, sum, 1);
    sum += __shfl_xor_sync(kFull, sum, 2);
    sum *= 0x1p-24f;
    q.sum[g][0] = __shfl_sync(kFull, sum, 8 * t);
    q.sum[g][1] = __shfl_sync(kFull, sum, 8 * t + 4);
  }
}

// Running state of a warp: columns are heads 2t, 2t + 1.
template <int D>
struct I4State {
  float o[D / 16][4];                 // O^T fragments, in units of 2^-24 (2^-20 for odd ones) / vmul
  float z[D / kInt4Group][2];         // this lane's part of sum p z
  float m[2], l[2];                   // reference maximum (log2 domain), this lane's part of sum p
  float vbound, vmul;                 // P~ = p s vmul, for s below vbound
};

template <typename T, int D, bool MASK>
__device__ __forceinline__ void i4_tile(uint32_t tile, int lo, int rows, const I4Query<D>& q, I4State<D>& st,
                                        int lane) {
  constexpr int GROUPS = D / kInt4Group;
  const int t = lane & 3, gr = lane >> 2;

  // S^T by groups: rows gr and gr + 8 of the tile.
  uint32_t kp0[GROUPS], kp1[GROUPS], vp0[GROUPS], vp1[GROUPS];
  lds_words<GROUPS>(tile + 16 * D + gr * (D / 16), kp0);
  lds_words<GROUPS>(tile + 16 * D + (gr + 8) * (D / 16), kp1);
  lds_words<GROUPS>(tile + 17 * D + gr * (D / 16), vp0);
  lds_words<GROUPS>(tile + 17 * D + (gr + 8) * (D / 16), vp1);
  constexpr int PER = D == 64 ? 2 : 4;  // words a shared load brings
  float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < D / 32 / PER; ++c) {
    uint32_t w0[PER], w1[PER];
    const int at = D == 256 ? 16 * ((4 * c + t) ^ (4 * (gr & 1))) : (D / 8) * t;
    lds_words<PER>(tile + gr * (D / 2) + at, w0);
    lds_words<PER>(tile + (gr + 8) * (D / 2) + at, w1);
#pragma unroll
    for (int h = 0; h < PER / 2; ++h) {
      const int g = c * (PER / 2) + h;
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t a[4], b[4];
        nibbles(w0[2 * h + i], a);
        nibbles(w1[2 * h + i], b);
        Mma<__half>::run(s, a[0], b[0], a[1], b[1], q.b[2 * (2 * g + i)][0], q.b[2 * (2 * g + i)][1]);
        Mma<__half>::run(s, a[2], b[2], a[3], b[3], q.b[2 * (2 * g + i) + 1][0], q.b[2 * (2 * g + i) + 1][1]);
      }
      const float2 k0 = pair_of<T>(kp0[g]), k1 = pair_of<T>(kp1[g]);
      x[0] = fmaf(s[0], k0.x, fmaf(k0.y, q.sum[g][0], x[0]));
      x[1] = fmaf(s[1], k0.x, fmaf(k0.y, q.sum[g][1], x[1]));
      x[2] = fmaf(s[2], k1.x, fmaf(k1.y, q.sum[g][0], x[2]));
      x[3] = fmaf(s[3], k1.x, fmaf(k1.y, q.sum[g][1], x[3]));
    }
  }
  float2 v0[GROUPS], v1[GROUPS];
  float smax = 0.f;
  bool on0 = true, on1 = true;
  if (MASK) {
    const int tok = 4 * (gr & 1) + (gr >> 1);  // the token of tile row gr (gr + 8: 8 more)
    on0 = tok >= lo && tok < rows;
    on1 = tok + 8 >= lo && tok + 8 < rows;
  }
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    v0[g] = MASK && !on0 ? make_float2(0.f, 0.f) : pair_of<T>(vp0[g]);
    v1[g] = MASK && !on1 ? make_float2(0.f, 0.f) : pair_of<T>(vp1[g]);
    smax = fmaxf(smax, fmaxf(v0[g].x, v1[g].x));
  }
  x[0] = on0 ? x[0] * q.mul[0] * 0x1p24f : -INFINITY;
  x[1] = on0 ? x[1] * q.mul[1] * 0x1p24f : -INFINITY;
  x[2] = on1 ? x[2] * q.mul[0] * 0x1p24f : -INFINITY;
  x[3] = on1 ? x[3] * q.mul[1] * 0x1p24f : -INFINITY;

  const float m0 = fmaxf(x[0], x[2]), m1 = fmaxf(x[1], x[3]);
  if (__any_sync(kFull, m0 > st.m[0] + kInt4Lazy || m1 > st.m[1] + kInt4Lazy || smax >= st.vbound)) {
    float n0 = m0, n1 = m1;
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      n0 = fmaxf(n0, __shfl_xor_sync(kFull, n0, off));
      n1 = fmaxf(n1, __shfl_xor_sync(kFull, n1, off));
      smax = fmaxf(smax, __shfl_xor_sync(kFull, smax, off));
    }
    float ratio = 1.f;
    if (smax >= st.vbound) {  // smax in [2^(E-1), 2^E): vbound = 2^E, vmul = 2^(7 - E)
      const int E = min(max(int((__float_as_uint(smax) >> 23) & 0xffu) - 126, -99), 126);
      const float mul = __uint_as_float(uint32_t(127 + 7 - E) << 23);
      ratio = mul / st.vmul;  // a power of two: exact
      st.vmul = mul;
      st.vbound = __uint_as_float(uint32_t(127 + E) << 23);
    }
    n0 = fmaxf(n0, st.m[0]);
    n1 = fmaxf(n1, st.m[1]);
    // a head without a score yet has nothing to rescale
    const float a0 = st.m[0] == -INFINITY ? 0.f : fast_exp2(st.m[0] - n0);
    const float a1 = st.m[1] == -INFINITY ? 0.f : fast_exp2(st.m[1] - n1);
    st.m[0] = n0;
    st.m[1] = n1;
    st.l[0] *= a0;
    st.l[1] *= a1;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      st.z[g][0] *= a0;
      st.z[g][1] *= a1;
    }
    const float r0 = a0 * ratio, r1 = a1 * ratio;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      st.o[i][0] *= r0;
      st.o[i][1] *= r1;
      st.o[i][2] *= r0;
      st.o[i][3] *= r1;
    }
  }
  // (a tile of nothing but -inf scores leaves the reference at -inf)
  const float ref0 = st.m[0] == -INFINITY ? 0.f : st.m[0], ref1 = st.m[1] == -INFINITY ? 0.f : st.m[1];
  float p[4] = {fast_exp2(x[0] - ref0), fast_exp2(x[1] - ref1), fast_exp2(x[2] - ref0), fast_exp2(x[3] - ref1)};
  st.l[0] += p[0] + p[2];
  st.l[1] += p[1] + p[3];
  uint32_t pb[GROUPS][2];
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    st.z[g][0] = fmaf(p[0], v0[g].y, fmaf(p[2], v1[g].y, st.z[g][0]));
    st.z[g][1] = fmaf(p[1], v0[g].y, fmaf(p[3], v1[g].y, st.z[g][1]));
    const float s0 = v0[g].x * st.vmul, s1 = v1[g].x * st.vmul;
    const __half2 h0 = __floats2half2_rn(p[0] * s0, p[1] * s0), h1 = __floats2half2_rn(p[2] * s1, p[3] * s1);
    pb[g][0] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h0));
    pb[g][1] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h1));
  }

  // O^T += C_V^T P~: K slot 2t + b + 8h is token 8h + 4b + t.
  const int turn = D == 64 ? 0 : D == 128 ? 4 * (t >> 1) : 2 * t;
  const uint32_t vt = tile + 8 * D + t * (D / 2) + (D / 16) * (gr ^ turn);
  uint32_t wa[GROUPS], wb[GROUPS], wc[GROUPS], wd[GROUPS];
  lds_words<GROUPS>(vt, wa);
  lds_words<GROUPS>(vt + 4 * (D / 2), wb);
  lds_words<GROUPS>(vt + 8 * (D / 2), wc);
  lds_words<GROUPS>(vt + 12 * (D / 2), wd);
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // nibbles 0..3, then 4..7
      uint32_t ab[4], cd[4];
      nibbles(__byte_perm(wa[g], wb[g], h ? 0x7632 : 0x5410), ab);
      nibbles(__byte_perm(wc[g], wd[g], h ? 0x7632 : 0x5410), cd);
      Mma<__half>::run(st.o[4 * g + 2 * h], ab[0], ab[2], cd[0], cd[2], pb[g][0], pb[g][1]);
      Mma<__half>::run(st.o[4 * g + 2 * h + 1], ab[1], ab[3], cd[1], cd[3], pb[g][0], pb[g][1]);
    }
  }
}

// Publishes a warp's (acc[G][D], m[G], l[G]) in head-dim order, powers of two
// taken out: row gr of fragment 4 g + 2 h + b is dim 64 g + 8 gr + 4 h + b, row
// gr + 8 the dim after the next.
template <int D, int G>
__device__ __forceinline__ void i4_publish(float* wsm, I4State<D>& st, int lane) {
  constexpr int GROUPS = D / kInt4Group;
  const int t = lane & 3, gr = lane >> 2;
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      st.l[c] += __shfl_xor_sync(kFull, st.l[c], off);
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) st.z[g][c] += __shfl_xor_sync(kFull, st.z[g][c], off);
    }
  }
  const float even = 0x1p24f / st.vmul, odd = 0x1p20f / st.vmul;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int head = 2 * t + c;
    if (head >= G) continue;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int dim = 64 * (i / 4) + 8 * gr + 4 * ((i / 2) & 1) + (i & 1);
      const float f = i & 1 ? odd : even;
      wsm[head * D + dim] = fmaf(st.o[i][c], f, st.z[i / 4][c]);
      wsm[head * D + dim + 2] = fmaf(st.o[i][2 + c], f, st.z[i / 4][c]);
    }
    if (gr == 0) {
      wsm[G * D + head] = st.m[c];
      wsm[G * D + G + head] = st.l[c];
    }
  }
}

template <typename T, int D, int G, int NW, int STAGES>
__global__ void __launch_bounds__(NW * 32) paged_decode_int4_kernel(const DecodeArgs a) {
  using C = I4Cfg<D, NW, STAGES>;
  static_assert(size_t(2 * G + G * D) * 4 <= size_t(STAGES) * C::TILE_BYTES, "merge area fits the ring");
  extern __shared__ __align__(128) unsigned char smem[];
  wait_for_predecessor();
  const int g = blockIdx.x, part = blockIdx.z;
  const int s = long_first_seq<NW>(a, blockIdx.y);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hq0 = g * a.group;

  // Without a window the first 32 block ids of this warp's tiles do not depend
  // on the length: read them together with it.
  int ids_early = 0;
  if (a.window == 0) {
    const int j0 = (part * a.part_tokens) / kBlock + warp + lane * NW;
    if (j0 < a.max_blocks_per_seq) ids_early = __ldg(a.block_tables + size_t(s) * a.max_blocks_per_seq + j0);
  }
  int L = a.context_lens[s];
  const int max_len = a.max_blocks_per_seq * kBlock;
  if (L < 0 || L > max_len) {
    if (threadIdx.x == 0 && part == 0 && g == 0) flag(a.status, PKV_DEV_BAD_CONTEXT_LEN);
    L = L < 0 ? 0 : max_len;
  }
  const TokenRange tr = token_range(L, a.window);
  const int nparts = L == 0 ? 1 : (L - tr.aligned + a.part_tokens - 1) / a.part_tokens;
  if (part >= nparts) return;
  if (L == 0) {
    T* o = static_cast<T*>(a.out) + (size_t(s) * a.num_q_heads + hq0) * D;
    for (int i = threadIdx.x; i < a.group * D / 8; i += NW * 32)
      reinterpret_cast<uint4*>(o)[i] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int t0 = tr.aligned + part * a.part_tokens;
  const int ntok = min(L, t0 + a.part_tokens) - t0;
  const int nb = (ntok + kBlock - 1) / kBlock;
  const int head = part == 0 ? tr.first - tr.aligned : 0;

  unsigned char* ring = smem + size_t(warp) * STAGES * C::TILE_BYTES;
  const uint32_t ring_s = smem_addr(ring);
  const uint32_t bar_s = smem_addr(smem + C::RING_BYTES) + warp * STAGES * 8;
  if (lane == 0) {
#pragma unroll
    for (int st = 0; st < STAGES; ++st) mbar_init(bar_s + 8 * st, 1);
    mbar_init_fence();
  }
  __syncwarp();

  const int n_my = nb > warp ? (nb - warp + NW - 1) / NW : 0;
  const int32_t* trow = a.block_tables + size_t(s) * a.max_blocks_per_seq + t0 / kBlock;
  auto checked = [&](int id) {
    if (id >= 0 && id < a.num_blocks) return id;
    flag(a.status, PKV_DEV_BAD_BLOCK_ID);
    return 0;
  };
  auto load_ids = [&](int batch) -> int {
    const int k = batch * 32 + lane;
    return k < n_my ? checked(__ldg(trow + warp + k * NW)) : 0;
  };
  int ids = lane < n_my ? checked(a.window == 0 ? ids_early : __ldg(trow + warp + lane * NW)) : 0;
  int ids_next = n_my > 32 ? load_ids(1) : 0;
  int id_batch = 0;
  const unsigned char* base = static_cast<const unsigned char*>(a.k_pool) + size_t(g) * C::TILE_BYTES;
  const size_t block_stride = size_t(a.num_kv_heads) * C::TILE_BYTES;
  auto issue = [&](int k) {  // warp-uniform; k increases by one per call
    if ((k >> 5) != id_batch) {
      ids = ids_next;
      ++id_batch;
      ids_next = (id_batch + 1) * 32 < n_my ? load_ids(id_batch + 1) : 0;
    }
    const int id = __shfl_sync(kFull, ids, k & 31);
    if (lane == 0) {
      const int st = k % STAGES;
      mbar_arrive_expect_tx(bar_s + 8 * st, C::TILE_BYTES);
      bulk_g2s(ring_s + st * C::TILE_BYTES, base + size_t(id) * block_stride, C::TILE_BYTES, bar_s + 8 * st);
    }
  };
  const int pre = n_my < STAGES ? n_my : STAGES;
  for (int k = 0; k < pre; ++k) issue(k);

  I4Query<D> q;
  i4_query<T, D>((lane >> 2) < a.group
                     ? static_cast<const T*>(a.q) + (size_t(s) * a.num_q_heads + hq0 + (lane >> 2)) * D
                     : nullptr,
                 lane, a.scale_log2, q);
  I4State<D> st;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
#pragma unroll
  for (int i = 0; i < C::GROUPS; ++i) st.z[i][0] = st.z[i][1] = 0.f;
  st.m[0] = st.m[1] = -INFINITY;
  st.l[0] = st.l[1] = 0.f;
  st.vbound = 0x1p-98f;
  st.vmul = 0x1p105f;

  for (int k = 0; k < n_my; ++k) {
    const int stage = k % STAGES;
    const bool ok = mbar_wait_bounded(bar_s + 8 * stage, (k / STAGES) & 1);
    if (!__all_sync(kFull, ok)) {
      // a copy never completed: record it, wait (bounded) for the others in flight, stop consuming
      if (lane == 0) flag(a.status, PKV_DEV_WAIT_TIMEOUT);
      const int last = min(n_my, k + STAGES);
      for (int kk = k; kk < last; ++kk) mbar_wait_bounded(bar_s + 8 * (kk % STAGES), (kk / STAGES) & 1);
      break;
    }
    const int j = warp + k * NW;
    const int rows = min(kBlock, ntok - j * kBlock);
    const int lo = j == 0 ? head : 0;
    const uint32_t tile = ring_s + stage * C::TILE_BYTES;
    if (rows == kBlock && lo == 0)
      i4_tile<T, D, false>(tile, 0, rows, q, st, lane);
    else
      i4_tile<T, D, true>(tile, lo, rows, q, st, lane);
    __syncwarp();
    if (k + STAGES < n_my) issue(k + STAGES);
  }
  i4_publish<D, G>(reinterpret_cast<float*>(ring), st, lane);
  __syncthreads();
  finish_chunk<T, D, G, NW>(a, smem, size_t(STAGES) * C::TILE_BYTES, s, g, part, nparts);
}

}  // namespace pkv
