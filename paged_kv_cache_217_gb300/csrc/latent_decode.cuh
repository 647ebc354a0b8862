// Latent attention decode (absorbed form) on the 5th-generation tensor cores.
//
// Every head h of a sequence attends over the same rows [c_p, r_p] (512 latent
// and 64 rotary elements):
//     x_hp = scale q_h . [c_p, r_p],   out_h = sum_p softmax(x_h)_p c_p,
// so a row is read once for all heads and used twice, as key and as value:
// 2 (576 + 512) operations per head and 1152 bytes per token.
//
// One CTA (1 per SM) takes up to N = 16, 32 or 64 heads and a range of 64-token
// tiles; both products run transposed, heads on the MMA's N:
//  * S^T[64 tokens, N] = K Q^T: A the tile's rows as they lie in shared memory
//    (K-major, 128-byte swizzle), B the queries (loaded once per sequence);
//  * O^T[512, N] += V^T P^T: A the same rows read along the other axis
//    (MN-major), 4 products of 128 dims per 16 tokens, B the weights P (16
//    bits, [N, 64]).
// With heads on M instead, O would need all 512 columns of tensor memory and
// leave none for S; transposed it takes 4 N columns, and S^T 2 N (two buffers).
// A tile arrives in thirds of 192 elements (3 chunks of 64), each by 4 TMA copies
// (one a 16-token block) of a 4-D view of the cache {64 elements, 8 rows, 9
// chunks, 8-row groups}, which lays a third out as groups of 3 swizzle atoms of 8
// rows x 128 bytes: both products step over tokens in strides of 3 KB and over
// elements in strides of 1 KB. Blocks past the end read the zero fill. The ring
// holds two tiles; O^T runs dims outermost, so that a third's place is free, and
// its next copy under way, while the product still reads the others, and S^T
// starts on the third that has landed. (Whole blocks at a time, freed by tokens,
// took 64.6 us for 32 sequences x 4000 tokens x 128 heads against 62.6; 36 copies
// of 16 x 64 boxes a tile took one warp 2700 cycles to issue.)
//
// Warps: 0-7 softmax and output (two of every quarter of tensor memory's lanes,
// each with half of the heads), 8 copies, 9 MMA issue. The MMA warp issues S^T of
// the next tile as its thirds land, and O^T of the current one as soon as its
// weights are there, also in the middle of that S^T: the softmax of tile i
// overlaps S^T of tile i + 1. An MMA reads both operands from shared memory at
// 128 bytes a cycle: S^T's M 64 takes 32 cycles at N 64, O^T's M 128 48; with the
// copies' writes a tile costs 2500 cycles of shared memory there, and a CTA
// measures 2600 a tile, which bounds 64 heads a CTA. With 16 heads (1450 cycles
// of products a tile) the cache's bytes bound it.
// The running maximum is a reference that moves only when a score exceeds it
// by 2^8 (one vote a tile); moving it rescales O^T in tensor memory. Weights
// are rounded to the cache's type (bf16: 2^-8 relative, one per weight). Their sum,
// in fp32, is of the rounded ones, so that the error is that of a weighted mean:
// delta_t p_t (c_t - out), nothing where one token has all the weight or the rows
// are alike.
//
// Work: the batch's tiles are one list cut into equal ranges, one per CTA (per
// block of heads), whatever the lengths. A sequence inside one range is written
// directly; the pieces of one that crosses ranges go to the workspace as fp32
// (max, sum, O) and latent_merge_kernel joins them by log-sum-exp.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "decode_mma.cuh"
#include "device_common.cuh"
#include "even_split.cuh"
#include "launch.h"

namespace pkv {

constexpr int kLatentSms = 152;       // CTAs a wave holds (one per SM of a GB300)
constexpr int kLatentTile = 64;       // tokens per tile
constexpr int kLatentSoftmax = 256;   // threads of the softmax warps
constexpr int kLatentThreads = kLatentSoftmax + 64;
constexpr float kLatentLazy = 8.f;
// fp16 weights are 2^7 times as large, 2^(7 + 8) at most: one 2^-21 of the largest still
// has all its bits (2^-14 without), and what fp16 loses of smaller ones is at most 2^-32
// of the largest. bf16 reaches far enough as it is.
constexpr float kLatentHeadroom = 7.f;
// Tiles between a copy and the prefetch of a later one into L2. 1: 46.9 us for 96
// sequences x 1500 tokens x 16 heads, 63.3 for 32 x 4000 x 128 (2: 47.9, 63.3; 4:
// 53.1, 64.4; none: 47.7, 67.7).
constexpr int kLatentAhead = 1;
constexpr int kLatentAtom = 1024;                 // 8 rows x 128 bytes
constexpr int kLatentGroup = 3 * kLatentAtom;     // 8 tokens of a third
constexpr int kLatentThird = 8 * kLatentGroup;    // 64 tokens x 192 elements
constexpr int kLatentTileBytes = 3 * kLatentThird;
// Offset of chunk c (64 elements) of a tile.
__host__ __device__ constexpr int latent_chunk(int c) { return c / 3 * kLatentThird + c % 3 * kLatentAtom; }

// Descriptors of the sequences that cross ranges: one per sequence {first range,
// last range} where there are at most as many sequences as ranges, else one per
// range {sequence that starts in it and goes on, last range}; -1: none.
inline size_t latent_desc_bytes(int ranges) { return (size_t(ranges) * sizeof(int2) + 15) / 16 * 16; }

template <int N>
struct LatentCfg {
  static constexpr int Q_BYTES = N * kLatentRow * 2;
  static constexpr int P_BYTES = N * kLatentTile * 2;
  static constexpr int MISC = 2048;  // barriers, statistics
  static constexpr size_t SMEM_BYTES = 1024 + MISC + Q_BYTES + P_BYTES + 2 * kLatentTileBytes;
  static constexpr int TMEM_COLS = 8 * N;  // 4 N for O^T, 2 N for S^T, a power of two
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

// ---- tcgen05 ----------------------------------------------------------------
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// Shared-memory matrix descriptor, 128-byte swizzle: start address, leading and
// stride byte offsets in 16-byte units, version 1, layout 2.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((addr >> 4) & 0x3fffu) | (uint64_t(lbo >> 4) << 16) | (uint64_t(sbo >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
// Instruction descriptor of kind::f16: fp32 accumulator, A and B of T, A
// MN-major when a_mn.
template <typename T>
__device__ constexpr uint32_t tc_idesc(int m, int n, bool a_mn) {
  const uint32_t type = sizeof(T) == 2 && !std::is_same<T, __half>::value ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | (uint32_t(a_mn) << 15) | (uint32_t(n >> 3) << 17) |
         (uint32_t(m >> 4) << 24);
}

// 16 lanes x 16 columns: thread l holds rows l / 4 and l / 4 + 8, columns
// 2 (l % 4), + 1 of each 8 (the layout of an mma.sync accumulator).
__device__ __forceinline__ void tc_ld_16x16(uint32_t addr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
               : "r"(addr));
}
// 32 lanes (one a thread) x 8 columns.
__device__ __forceinline__ void tc_ld_32x8(uint32_t addr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
               : "r"(addr));
}
__device__ __forceinline__ void tc_st_32x8(uint32_t addr, const float* r) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(u[0]),
               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void l2_prefetch(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// A look at a barrier's phase, without the wait that try_wait may take.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void stsm_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}
// One lane of a converged warp. The compiler knows that a branch on it is taken
// by one lane: tcgen05.mma's operands then stay in uniform registers (a branch
// on the lane index issued one MMA in 155 cycles, this one in 23 to 48).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// 16 lanes x 8 columns.
__device__ __forceinline__ void tc_ld_16x8(uint32_t addr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
               : "r"(addr));
}
__device__ __forceinline__ void stsm_x2_trans(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// Barrier of the four softmax warps of one half of the heads.
__device__ __forceinline__ void softmax_sync(int half) { asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory"); }
__device__ __forceinline__ bool softmax_any(int half, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbar.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + half), "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// ---- work -------------------------------------------------------------------
__device__ __forceinline__ int latent_len(const LatentArgs& a, int s) {
  const int L = a.context_lens[s], most = a.max_blocks_per_seq * kBlock;
  return L < 0 ? 0 : L > most ? most : L;
}
__device__ __forceinline__ int latent_tiles(int L) { return (L + kLatentTile - 1) / kLatentTile; }

// Shared state of a CTA outside the operand buffers.
template <int N>
struct LatentShared {
  uint64_t third_full[6], third_empty[6];    // slot 0's thirds, slot 1's
  uint64_t q_full, q_empty, s_full[2], p_full, pv_done;
  uint32_t tmem;
  int stop;  // a wait gave up: every role leaves
  int first_seq, first_len;
  long long first_tile;                      // list index of first_seq's first tile
  long long scan[kLatentThreads / 32];
  uint64_t drain;                            // after a wait gave up
  float stat[4][N], alpha[N], mref[N];       // per warp and head; rescale factors; references
};

// Waits for a phase; false when the limit ran out or another role gave up.
__device__ __forceinline__ bool latent_wait(uint32_t bar, uint32_t parity, volatile int* stop, unsigned int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*stop) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      *stop = 1;
      flag(status, PKV_DEV_WAIT_TIMEOUT);
      return false;
    }
  }
  return true;
}

// Walks a CTA's range [begin, end) of the tile list as segments of one sequence.
// The next sequence's length is read one segment ahead.
struct LatentWalk {
  int s;                    // sequence
  int L, ahead;             // its length, and the next sequence's
  long long at, end;        // list index of the next segment's first tile, and the range's end
  long long base;           // list index of sequence s's first tile
  int first, last, n;       // the segment: its tiles [first, last) of the n of the sequence
  __device__ __forceinline__ void start(const LatentArgs& a, int seq, int len, long long tile0, long long b,
                                        long long e) {
    s = seq;
    base = tile0;
    at = b;
    end = e;
    L = len;
    ahead = b < e && s + 1 < a.num_seqs ? latent_len(a, s + 1) : 0;
  }
  __device__ __forceinline__ bool next(const LatentArgs& a) {
    if (at >= end) return false;
    while (base + (n = latent_tiles(L)) <= at) {
      base += n;
      ++s;
      L = ahead;
      ahead = s + 1 < a.num_seqs ? latent_len(a, s + 1) : 0;
    }
    first = int(at - base);
    last = base + n < end ? n : int(end - base);
    at = base + last;
    return true;
  }
};

template <typename T, int N>
__global__ void __launch_bounds__(kLatentThreads, 1)
latent_decode_kernel(const LatentArgs a, const __grid_constant__ CUtensorMap cache_map,
                     const __grid_constant__ CUtensorMap q_map) {
  using C = LatentCfg<N>;
  static_assert(sizeof(LatentShared<N>) <= C::MISC, "shared state");
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem) + 1023) & ~uintptr_t(1023));
  unsigned char* q_mem = base;                       // 9 chunks of [N][64]
  unsigned char* p_mem = q_mem + C::Q_BYTES;         // [N][64 tokens]
  unsigned char* ring = p_mem + C::P_BYTES;          // two tiles
  LatentShared<N>& sh = *reinterpret_cast<LatentShared<N>*>(ring + 2 * kLatentTileBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hb = int(blockIdx.x) % a.head_blocks, range = int(blockIdx.x) / a.head_blocks;
  const int h0 = hb * a.block_heads, heads = min(a.block_heads, a.num_heads - h0);

  if (tid == 0) {
    for (int i = 0; i < 6; ++i) {
      mbar_init(smem_addr(&sh.third_full[i]), 1);
      mbar_init(smem_addr(&sh.third_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(smem_addr(&sh.s_full[i]), 1);
    mbar_init(smem_addr(&sh.q_full), 1);
    mbar_init(smem_addr(&sh.q_empty), 1);
    mbar_init(smem_addr(&sh.p_full), kLatentSoftmax);
    mbar_init(smem_addr(&sh.pv_done), 1);
    mbar_init_fence();
    sh.stop = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&cache_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&q_map) : "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                 "r"(uint32_t(C::TMEM_COLS))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // The tables' way into L2 begins while the lengths are read (tables of up to 1
  // MB: a line a thread).
  const size_t line = size_t(blockIdx.x * unsigned(kLatentThreads) + tid) * 32;
  const size_t ids_held = size_t(a.num_seqs) * a.max_blocks_per_seq;
  if (ids_held <= (1u << 18) && line < ids_held)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.block_tables + line));
  // The tile list: each thread sums a run of sequences, a scan of the sums
  // gives every run's place in the list, and the thread whose run holds this
  // range's first tile finds its sequence.
  const int per = (a.num_seqs + kLatentThreads - 1) / kLatentThreads;
  const int run0 = min(a.num_seqs, tid * per), run1 = min(a.num_seqs, run0 + per);
  int zero_len = int(blockIdx.x) < a.num_seqs ? latent_len(a, int(blockIdx.x)) : 1;  // (read along with the others)
  long long mine = 0;
  int len = 0;  // of the run's last sequence
  for (int s = run0; s < run1; ++s) {
    const int raw = a.context_lens[s], most = a.max_blocks_per_seq * kBlock;
    if ((raw < 0 || raw > most) && blockIdx.x == 0) flag(a.status, PKV_DEV_BAD_CONTEXT_LEN);
    len = raw < 0 ? 0 : raw > most ? most : raw;
    mine += latent_tiles(len);
  }
  long long upto = mine;  // inclusive scan over the warp, then over the warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(kFull, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) sh.scan[warp] = upto;
  __syncthreads();
  long long before = upto - mine, total = 0;
#pragma unroll
  for (int i = 0; i < kLatentThreads / 32; ++i) {
    if (i < warp) before += sh.scan[i];
    total += sh.scan[i];
  }
  const int used = total < a.ranges ? int(total) : a.ranges;  // ranges that get tiles
  const EvenSplit split(total, used > 0 ? used : 1);
  const long long begin = range < used ? split.begin(range) : 0, end = range < used ? split.begin(range + 1) : 0;
  if (begin < end && begin >= before && begin < before + mine) {
    long long at = before;
    int s = run0;
    if (per > 1) {
      for (;; ++s) {
        len = latent_len(a, s);
        if (at + latent_tiles(len) > begin) break;
        at += latent_tiles(len);
      }
    }
    sh.first_seq = s;
    sh.first_len = len;
    sh.first_tile = at;
  }
  // Sequences without tokens: zeros, spread over the CTAs.
  for (int s = int(blockIdx.x); s < a.num_seqs;) {
    if (zero_len == 0) {
      uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + size_t(s) * a.num_heads * kLatentDim);
      for (int i = tid; i < a.num_heads * kLatentDim / 8; i += kLatentThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
      if (tid == 0 && a.desc_by_seq) a.desc[s] = make_int2(-1, 0);
    }
    s += int(gridDim.x);
    if (s < a.num_seqs) zero_len = latent_len(a, s);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  LatentWalk walk;
  walk.start(a, sh.first_seq, sh.first_len, sh.first_tile, begin, end);
  volatile int* stop = &sh.stop;
  bool open = false;  // (thread 0) the range's last sequence starts in it and goes on past it

  if (warp == 8) {
    // ---- copies ----
    int tile = 0, seg = 0;
    int next_seq = -1, next_ids = 0;
    bool ok = true;  // warp-uniform
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
      return bool(__all_sync(kFull, latent_wait(bar, parity, stop, a.status)));
    };
    while (ok && walk.next(a)) {
      // Block ids of the segment, 32 at a time and the next 32 ahead: lane l of
      // `ids` holds the id of block ids_from + l, of `ids_ahead` the one 32 on.
      // Blocks past the end name rows outside the tensor, which read as zeros.
      const int nb = (walk.L + kBlock - 1) / kBlock;
      const int32_t* row = a.block_tables + size_t(walk.s) * a.max_blocks_per_seq;
      auto load_ids = [&](int from) {
        const int j = from + lane;
        return j < nb ? row[j] : a.num_blocks;
      };
      auto checked = [&](int id, int j) {
        if (id >= 0 && (id < a.num_blocks || j >= nb)) return id;
        flag(a.status, PKV_DEV_BAD_BLOCK_ID);
        return 0;
      };
      int ids_from = 4 * walk.first;
      int ids = next_seq == walk.s && ids_from == 0 ? (lane < nb ? next_ids : a.num_blocks) : load_ids(ids_from);
      int ids_ahead = load_ids(ids_from + 32);
      // the queries, while the ids are on their way
      if (seg > 0) ok = wait_all(smem_addr(&sh.q_empty), (seg - 1) & 1);
      if (!ok) break;
      if (elect_one()) {
        const uint32_t qb = smem_addr(&sh.q_full);
        mbar_arrive_expect_tx(qb, C::Q_BYTES);
        tma_load_4d(smem_addr(q_mem), &q_map, 0, h0, 0, walk.s, qb);
      }
      ++seg;
      ids = checked(ids, ids_from + lane);
      // the next sequence's first ids, for its rows' way into L2
      next_seq = walk.s + 1;
      next_ids = next_seq < a.num_seqs && lane < a.max_blocks_per_seq
                     ? a.block_tables[size_t(next_seq) * a.max_blocks_per_seq + lane]
                     : 0;
      const int next_nb = walk.at < walk.end && next_seq < a.num_seqs ? (walk.ahead + kBlock - 1) / kBlock : 0;
      for (int t = walk.first; ok && t < walk.last; ++t, ++tile) {
        if (4 * t >= ids_from + 32) {
          ids_from += 32;
          ids = checked(ids_ahead, ids_from + lane);
          ids_ahead = load_ids(ids_from + 32);
        }
        // ids of the tile, and of the one kLatentAhead on (-1: none)
        int id[4], far_id[4];
        const int over = t + kLatentAhead - walk.last, far = 4 * (t + kLatentAhead) - ids_from;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          id[j] = __shfl_sync(kFull, ids, 4 * t - ids_from + j);
          const int x = __shfl_sync(kFull, over >= 0 ? next_ids : far < 32 ? ids : ids_ahead,
                                    (over >= 0 ? 4 * over + j : far + j) & 31);
          far_id[j] = x < a.num_blocks && (over < 0 || 4 * over + j < next_nb) ? x : -1;
        }
        if (elect_one()) {
          const uint32_t fb = smem_addr(&sh.third_full[3 * (tile & 1)]), eb = smem_addr(&sh.third_empty[3 * (tile & 1)]);
          const uint32_t dst = smem_addr(ring) + (tile & 1) * kLatentTileBytes;
          bool go = true;
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            if (tile >= 2) go = go && latent_wait(eb + 8 * c, ((tile >> 1) - 1) & 1, stop, a.status);
            // (announced only now: third_empty says that the last use's copies,
            // and with them that phase of third_full, are over)
            if (!go) break;
            mbar_arrive_expect_tx(fb + 8 * c, kLatentThird);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tma_load_4d(dst + c * kLatentThird + j * (2 * kLatentGroup), &cache_map, 0, 0, 3 * c, 2 * id[j], fb + 8 * c);
          }
          // rows that a later copy takes start their way into L2 now, so that the
          // copy, issued when a place is free, waits for L2 only
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (far_id[j] >= 0)
              l2_prefetch(static_cast<const T*>(a.cache) + size_t(far_id[j]) * (kBlock * kLatentRow),
                          kBlock * kLatentRow * sizeof(T));
        }
        __syncwarp();
        ok = !*stop;
        ok = __all_sync(kFull, ok);
      }
    }
    if (*stop) {
      // Wait (bounded) for the copies in flight. A tile whose copies were not
      // all issued never completes its phase: its wait runs to the limit.
      for (int i = 0; i < 2; ++i) {
        const int uses = tile >= i ? (tile - i) / 2 + 1 : 0;
        if (uses > 0)
          for (int c = 0; c < 3; ++c)
            mbar_wait_bounded(smem_addr(&sh.third_full[3 * i + c]), (uses - 1) & 1, 10000000ull);
      }
      if (seg > 0) mbar_wait_bounded(smem_addr(&sh.q_full), (seg - 1) & 1, 10000000ull);
    }
  } else if (warp == 9) {
    // ---- MMA issue: one lane ----
    if (elect_one()) {
      constexpr uint32_t id_s = tc_idesc<T>(kLatentTile, N, false), id_o = tc_idesc<T>(128, N, true);
      const uint64_t q_desc = tc_desc(smem_addr(q_mem), 16, 1024), p_desc = tc_desc(smem_addr(p_mem), 16, 1024);
      const uint64_t key_desc = tc_desc(smem_addr(ring), 16, kLatentGroup);
      uint64_t val_desc[4];  // dims 128 j .. + 127: chunks 2 j and 2 j + 1
#pragma unroll
      for (int j = 0; j < 4; ++j)
        val_desc[j] = tc_desc(smem_addr(ring) + latent_chunk(2 * j), latent_chunk(2 * j + 1) - latent_chunk(2 * j), kLatentGroup);
      const int n = int(end - begin);
      int qk = 0, pv = 0, seg = 0;      // tiles whose S^T, O^T are issued; segments whose queries are waited for
      bool seg_first = true;            // tile qk starts a segment
      uint32_t starts = 0;              // bit t & 1: tile t starts a segment (t = pv, pv + 1)
      int t = 0;                        // tile qk within its sequence
      if (n > 0) {
        walk.next(a);
        t = walk.first;
      }
      // O^T of tile pv, if its weights are there
      auto outputs = [&]() {
        if (pv >= qk || !mbar_test(smem_addr(&sh.p_full), pv & 1)) return false;
        tc_fence_after();
        const uint32_t at = (pv & 1) * (kLatentTileBytes >> 4);
        const bool first = (starts >> (pv & 1)) & 1u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {    // 128 dims
#pragma unroll
          for (int k = 0; k < 4; ++k)    // 16 tokens
            tc_mma(tmem + j * N, val_desc[j] + at + k * (2 * kLatentGroup >> 4), p_desc + 2 * k, id_o, !(first && k == 0));
          if (j > 0) tc_commit(smem_addr(&sh.third_empty[3 * (pv & 1) + j - 1]));  // (its last chunk is 3 j - 1)
        }
        tc_commit(smem_addr(&sh.pv_done));
        ++pv;
        return true;
      };
      // Waits, for a limited time, until done() says so, and issues O^T meanwhile.
      auto until = [&](auto done) {
        unsigned long long t0 = 0;
        for (int polls = 0; !done(); ++polls) {
          if (outputs()) polls = 0;
          if ((polls & 63) != 63) continue;
          const unsigned long long now = global_timer_ns();
          if (polls == 63) t0 = now;
          if (*stop) return false;
          if (now - t0 > kWaitLimitNs) {
            *stop = 1;
            flag(a.status, PKV_DEV_WAIT_TIMEOUT);
            return false;
          }
        }
        return true;
      };
      bool ok = true;
      while (ok && qk < n) {
        // S^T's buffer is free once tile qk - 2 has its weights
        ok = until([&]() { return qk < pv + 2; });
        if (ok && seg_first) ok = until([&]() { return mbar_test(smem_addr(&sh.q_full), seg & 1); });
        const uint32_t d = tmem + 4 * N + (qk & 1) * N, full = smem_addr(&sh.third_full[3 * (qk & 1)]);
        const uint64_t key = key_desc + (qk & 1) * (kLatentTileBytes >> 4);
#pragma unroll
        for (int c = 0; c < kLatentRow / 64; ++c) {
          if (c >= 3 && c <= 7) outputs();
          if (c % 3 == 0) {
            ok = ok && until([&]() { return mbar_test(full + 8 * (c / 3), (qk >> 1) & 1); });
            if (!ok) break;
            tc_fence_after();
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma(d, key + (latent_chunk(c) >> 4) + 2 * k, q_desc + c * (N * 128 >> 4) + 2 * k, id_s, c + k > 0);
        }
        if (!ok) break;
        tc_commit(smem_addr(&sh.s_full[qk & 1]));
        starts = (starts & ~(1u << (qk & 1))) | (uint32_t(seg_first) << (qk & 1));
        seg += seg_first ? 1 : 0;
        seg_first = ++t == walk.last;
        if (seg_first) {
          tc_commit(smem_addr(&sh.q_empty));
          if (walk.next(a)) t = walk.first;
        }
        ++qk;
      }
      if (ok) until([&]() { return pv == n; });
      if (*stop) {  // let the products in flight end before the tensor memory is freed
        const uint32_t bar = smem_addr(&sh.drain);
        mbar_init(bar, 1);
        mbar_init_fence();
        tc_commit(bar);
        mbar_wait_bounded(bar, 0, 10000000ull);
      }
    }
    __syncwarp();
  } else {
    // ---- softmax and output ----
    // Warps w and w + 4 read lanes 32 (w % 4) .. of tensor memory (tokens 16 (w %
    // 4) .. + 15 of S^T, dims 32 (w % 4) .. + 31 of each product of O^T), for
    // heads HALF (w / 4) .. . This thread keeps heads 8 i + 2 t, + 1 of its half.
    constexpr int HALF = N / 2, G8 = HALF / 8;
    constexpr float kHeadroom = std::is_same<T, __half>::value ? kLatentHeadroom : 0.f;
    const int t = lane & 3, gr = lane >> 2, quarter = warp & 3, half = warp >> 2, hs = half * HALF;
    const uint32_t lanes = uint32_t(quarter * 32) << 16;
    // (After a wait gave up, `stop` lets every later wait return at once: these
    // warps then run out their loops, together and without further waiting.)
    int tile = 0;
    while (walk.next(a)) {
      float m[G8][2], l[G8][2];
#pragma unroll
      for (int i = 0; i < G8; ++i) m[i][0] = m[i][1] = -INFINITY, l[i][0] = l[i][1] = 0.f;
      for (int u = walk.first; u < walk.last; ++u, ++tile) {
        latent_wait(smem_addr(&sh.s_full[tile & 1]), (tile >> 1) & 1, stop, a.status);
        tc_fence_after();
        float x[G8][4];  // rows gr (0, 1) and gr + 8 (2, 3) of this warp's 16 tokens
        const uint32_t s_at = tmem + lanes + 4 * N + (tile & 1) * N + hs;
        if constexpr (G8 == 1) {
          tc_ld_16x8(s_at, &x[0][0]);
        } else {
#pragma unroll
          for (int i = 0; i < G8; i += 2) tc_ld_16x16(s_at + 8 * i, &x[i][0]);
        }
        tc_wait_ld();
        const int left = walk.L - u * kLatentTile;  // tokens of this tile
        const bool on0 = 16 * quarter + gr < left, on1 = 16 * quarter + gr + 8 < left;
        bool move = false;
#pragma unroll
        for (int i = 0; i < G8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[i][e] = on0 ? x[i][e] * a.scale_log2 : -INFINITY;
            x[i][2 + e] = on1 ? x[i][2 + e] * a.scale_log2 : -INFINITY;
            move |= fmaxf(x[i][e], x[i][2 + e]) > m[i][e] + kLatentLazy;
          }
        const bool moving = softmax_any(half, move);
        if (moving) {
#pragma unroll
          for (int i = 0; i < G8; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = fmaxf(x[i][e], x[i][2 + e]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
              if (gr == 0) sh.stat[quarter][hs + 8 * i + 2 * t + e] = v;
            }
          softmax_sync(half);
#pragma unroll
          for (int i = 0; i < G8; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int h = hs + 8 * i + 2 * t + e;
              const float v = fmaxf(fmaxf(fmaxf(sh.stat[0][h], sh.stat[1][h]), fmaxf(sh.stat[2][h], sh.stat[3][h])),
                                    m[i][e]);
              // a head without a score yet has nothing to rescale
              const float al = m[i][e] == -INFINITY ? 0.f : fast_exp2(m[i][e] - v);
              m[i][e] = v;
              l[i][e] *= al;
              if (quarter == 0 && gr == 0) sh.alpha[h] = al;
            }
          softmax_sync(half);
        }
        uint32_t p[G8][2];  // weights of rows gr and gr + 8, two heads each
#pragma unroll
        for (int i = 0; i < G8; ++i) {
          const float ref0 = (m[i][0] == -INFINITY ? 0.f : m[i][0]) - kHeadroom;
          const float ref1 = (m[i][1] == -INFINITY ? 0.f : m[i][1]) - kHeadroom;
          p[i][0] = pack2<T>(fast_exp2(x[i][0] - ref0), fast_exp2(x[i][1] - ref1));
          p[i][1] = pack2<T>(fast_exp2(x[i][2] - ref0), fast_exp2(x[i][3] - ref1));
        }
        // P and O^T are free once the previous tile's product is done
        if (tile > 0) latent_wait(smem_addr(&sh.pv_done), (tile - 1) & 1, stop, a.status);
        if (moving && u > walk.first) {
          tc_fence_after();
#pragma unroll 1
          for (int j = 0; j < kLatentDim / 128; ++j) {
#pragma unroll
            for (int c = 0; c < HALF; c += 8) {
              float o[8];
              tc_ld_32x8(tmem + lanes + j * N + hs + c, o);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] *= sh.alpha[hs + c + i];
              tc_st_32x8(tmem + lanes + j * N + hs + c, o);
            }
          }
          tc_wait_st();
        }
        if (left < kLatentTile) {
          // rows past the end hold whatever the block holds (NaN included): as
          // values they must be zeros
          const int dead = min(kLatentTile, (left + kBlock - 1) / kBlock * kBlock) - left;
          for (int i = tid; i < dead * (kLatentDim / 8); i += kLatentSoftmax) {
            const int v = i % (kLatentDim / 8), r = left + i / (kLatentDim / 8);
            *reinterpret_cast<uint4*>(ring + (tile & 1) * kLatentTileBytes + latent_chunk(v / 8) + r / 8 * kLatentGroup +
                                      r % 8 * 128 + v % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        // P: row a head, 16-byte chunk 8 tokens. Matrix b = lane / 8: tokens 8 (b &
        // 1), heads 8 (i + b / 2); its row lane % 8 a head.
        const int b = lane >> 3, chunk = 2 * quarter + (b & 1);
        if constexpr (G8 == 1) {
          const int head = hs + (lane & 7);
          stsm_x2_trans(smem_addr(p_mem) + head * 128 + ((chunk ^ (head & 7)) << 4), p[0][0], p[0][1]);
        } else {
#pragma unroll
          for (int i = 0; i < G8; i += 2) {
            const int head = hs + 8 * (i + (b >> 1)) + (lane & 7);
            stsm_x4_trans(smem_addr(p_mem) + head * 128 + ((chunk ^ (head & 7)) << 4), p[i][0], p[i][1], p[i + 1][0],
                          p[i + 1][1]);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        mbar_arrive(smem_addr(&sh.p_full));
#pragma unroll
        for (int i = 0; i < G8; ++i) {
          const float2 a = unpack2<T>(p[i][0]), b = unpack2<T>(p[i][1]);
          l[i][0] += a.x + b.x;
          l[i][1] += a.y + b.y;
        }
      }
      // The segment's sums, then its output: thread = dim, columns = heads.
#pragma unroll
      for (int i = 0; i < G8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[i][e] += __shfl_xor_sync(kFull, l[i][e], o);
          if (gr == 0) {
            sh.stat[quarter][hs + 8 * i + 2 * t + e] = l[i][e];
            if (quarter == 0) sh.mref[hs + 8 * i + 2 * t + e] = m[i][e];
          }
        }
      const bool whole = walk.first == 0 && walk.last == walk.n;
      const int slot = 2 * range + (walk.first == 0 ? 1 : 0);
      softmax_sync(half);
      const int th = tid & 127;
      if (th < HALF) {
        const int h = hs + th;
        const float sum = (sh.stat[0][h] + sh.stat[1][h]) + (sh.stat[2][h] + sh.stat[3][h]);
        sh.alpha[h] = 1.f / sum;
        if (!whole) a.part_ml[(size_t(slot) * a.head_blocks + hb) * N + h] = make_float2(sh.mref[h], sum);
      }
      if (tid == 0 && hb == 0 && walk.first == 0) {
        // the ranges that hold the rest of this sequence: up to the one with its last tile
        int2 d = make_int2(-1, 0);
        if (!whole) {
          const int r = split.of(walk.base + walk.n - 1);
          d = a.desc_by_seq ? make_int2(range, r) : make_int2(walk.s, r);
          open = true;
        }
        if (a.desc_by_seq) a.desc[walk.s] = d;
        else if (!whole) a.desc[range] = d;
      }
      latent_wait(smem_addr(&sh.pv_done), (tile - 1) & 1, stop, a.status);
      softmax_sync(half);
      tc_fence_after();
      T* const out = static_cast<T*>(a.out) + (size_t(walk.s) * a.num_heads + h0 + hs) * kLatentDim;
      float* const part = a.part_o + ((size_t(slot) * a.head_blocks + hb) * N + hs) * kLatentDim + quarter * 32 + lane;
#pragma unroll 1
      for (int j = 0; j < kLatentDim / 128; ++j) {
        float o[2][8];
        tc_ld_32x8(tmem + lanes + j * N + hs, o[0]);
#pragma unroll
        for (int c = 0; c < HALF / 8; ++c) {
          tc_wait_ld();
          if (c + 1 < HALF / 8) tc_ld_32x8(tmem + lanes + j * N + hs + 8 * (c + 1), o[(c + 1) & 1]);
          float(&x)[8] = o[c & 1];
          if (whole) {
            // two heads a step: even lanes take the first one's dims lane, lane +
            // 1, odd lanes the second one's dims lane - 1, lane
            const int dim = j * 128 + quarter * 32 + (lane & ~1);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float e = x[i] * sh.alpha[hs + 8 * c + i], f = x[i + 1] * sh.alpha[hs + 8 * c + i + 1];
              const float g = __shfl_xor_sync(kFull, lane & 1 ? e : f, 1);
              const int h = 8 * c + i + (lane & 1);
              if (hs + h < heads)
                *reinterpret_cast<uint32_t*>(out + size_t(h) * kLatentDim + dim) =
                    lane & 1 ? pack2<T>(g, f) : pack2<T>(e, g);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) part[(8 * c + i) * kLatentDim + j * 128] = x[i];  // (padding heads too)
          }
        }
      }
      tc_fence_before();   // the next segment's O^T comes after these reads
      softmax_sync(half);  // statistics are read: the next segment may write them
    }
  }
  // A range without a sequence that goes on past it says so.
  if (tid == 0 && hb == 0) {
    if (!open && !a.desc_by_seq) a.desc[range] = make_int2(-1, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(uint32_t(C::TMEM_COLS)));
  }
}

// Joins the pieces of a sequence that crosses ranges:
// out = sum_i w_i o_i / sum_i w_i l_i with w_i = 2^(m_i - max m). A CTA takes two
// heads (one with Z = 4). Few pieces (at most kFewPieces): one round of loads,
// each half of the CTA a head, 4 dims per thread. Many: head after head -- the
// weights of all pieces, and 2 Z groups of threads each take every 2 Z-th piece,
// the first of them read while the weights are made; Z = 4 cuts the dims over 4
// CTAs (few heads in all).
constexpr int kFewPieces = 8;
template <typename T, int N, int Z>
__global__ void __launch_bounds__(256) latent_merge_kernel(const LatentArgs a) {
  constexpr int LANES = kLatentDim / 4 / Z, GROUPS = 256 / LANES;
  __shared__ float weight[kLatentSms], red[8];
  __shared__ float4 other[GROUPS - 1][LANES];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  const int2 desc = __ldcg(a.desc + blockIdx.x);
  if (desc.x < 0) return;
  const int r0 = a.desc_by_seq ? desc.x : int(blockIdx.x), s = a.desc_by_seq ? int(blockIdx.x) : desc.x;
  const int n = desc.y - r0 + 1;
  auto slot = [&](int i, int h) {
    const int hb = h / a.block_heads;
    return (size_t(2) * (r0 + i) + (i == 0 ? 1 : 0)) * a.head_blocks * N + hb * N + h - hb * a.block_heads;
  };
  auto write = [&](int h, int d, const float4& x, float den) {
    const float inv = 1.f / den;
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (size_t(s) * a.num_heads + h) * kLatentDim + d) =
        make_uint2(pack2<T>(x.x * inv, x.y * inv), pack2<T>(x.z * inv, x.w * inv));
  };
  if (Z == 1 && n <= kFewPieces) {
    const int h = 2 * int(blockIdx.y) + (tid >> 7), d = (tid & 127) * 4;
    if (h >= a.num_heads) return;
    float2 ml[kFewPieces];
    float4 o[kFewPieces];
    float M = -INFINITY;
#pragma unroll
    for (int i = 0; i < kFewPieces; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        ml[i] = __ldcg(a.part_ml + slot(i, h));
        o[i] = __ldcg(reinterpret_cast<const float4*>(a.part_o + slot(i, h) * kLatentDim + d));
      }
    }
#pragma unroll
    for (int i = 0; i < kFewPieces; ++i) M = fmaxf(M, ml[i].x);
    const float ref = M == -INFINITY ? 0.f : M;
    float den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kFewPieces; ++i) {
      const float w = fast_exp2(ml[i].x - ref);
      den = fmaf(w, ml[i].y, den);
      num.x = fmaf(w, o[i].x, num.x);
      num.y = fmaf(w, o[i].y, num.y);
      num.z = fmaf(w, o[i].z, num.z);
      num.w = fmaf(w, o[i].w, num.w);
    }
    write(h, d, num, den);
    return;
  }
  const int group = tid / LANES, d = (int(blockIdx.z) * LANES + tid % LANES) * 4;
  constexpr int HEADS = Z == 1 ? 2 : 1;
  constexpr int AHEAD = Z == 1 ? kFewPieces : (kLatentSms + GROUPS - 1) / GROUPS;  // pieces read while the weights are made
  for (int h = HEADS * int(blockIdx.y); h < min(a.num_heads, HEADS * int(blockIdx.y) + HEADS); ++h) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (tid < n) ml = __ldcg(a.part_ml + slot(tid, h));
    float4 early[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = group + k * GROUPS;
      early[k] = i < n ? __ldcg(reinterpret_cast<const float4*>(a.part_o + slot(i, h) * kLatentDim + d))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float M = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    __syncthreads();  // the last head's readers are done
    if ((tid & 31) == 0) red[tid >> 5] = M;
    __syncthreads();
    M = red[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) M = fmaxf(M, red[i]);
    const float w = tid < n ? fast_exp2(ml.x - (M == -INFINITY ? 0.f : M)) : 0.f;
    if (tid < n) weight[tid] = w;
    float den = w * ml.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(kFull, den, o);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = den;
    __syncthreads();
    den = red[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) den += red[i];
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int i, const float4& o) {
      const float wi = weight[i];
      num.x = fmaf(wi, o.x, num.x);
      num.y = fmaf(wi, o.y, num.y);
      num.z = fmaf(wi, o.z, num.z);
      num.w = fmaf(wi, o.w, num.w);
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (group + k * GROUPS < n) add(group + k * GROUPS, early[k]);
#pragma unroll 8
    for (int i = group + AHEAD * GROUPS; i < n; i += GROUPS)
      add(i, __ldcg(reinterpret_cast<const float4*>(a.part_o + slot(i, h) * kLatentDim + d)));
    if (group) other[group - 1][tid % LANES] = num;
    __syncthreads();
    if (group) continue;
#pragma unroll
    for (int i = 0; i < GROUPS - 1; ++i) {
      const float4 x = other[i][tid];
      num.x += x.x;
      num.y += x.y;
      num.z += x.z;
      num.w += x.w;
    }
    write(h, d, num, den);
  }
}

}  // namespace pkv
