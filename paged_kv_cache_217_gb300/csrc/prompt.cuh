// Attention of many query rows over the paged cache on the 5th-generation tensor
// cores: prompts, chunks of prompts and drafted tokens (causal), cross attention, and
// the decode of groups that share a prefix.
//
// A row is a (query token, query head) pair; the G heads of a KV head lie together, so
// that the K and V of a head are read once for all of them:
//     S = Q K^T (fp32),  p = 2^(scale log2(e) S - m),  O += P V,  l += sum p,  out = O / l.
// One CTA (1 per SM) takes pieces of items. An item is a block of up to 256 rows of one
// KV head (128 with head_dim 256) and the positions that any of them sees; a piece is
// some of its tiles of 64 tokens.
//
// Warps: two softmax warpgroups (a thread a row of the tile), one warp each that copies
// K and V and copies Q, and one for each warpgroup that issues its MMAs. Warpgroup w owns
// O_w (head_dim columns of tensor memory) and two S of 64 columns. A block of more than
// 128 rows gives each warpgroup a tile of rows and every K and V tile is used by both; of
// smaller ones a long piece gives both the same rows and every other tile, joined at its
// end, and short ones go to the warpgroups in turn. With head_dim 256 O leaves room for
// one warpgroup.
//  * S = Q K^T: both operands in shared memory, K-major, 128-byte swizzle.
//  * P overwrites S as 16-bit values, and is the A operand from there; V is read
//    MN-major from the tile as it lies.
// While a warpgroup works on its scores the tensor cores run the other's products and its
// own next scores. The running maximum is a reference that moves only when a score exceeds
// it by 2^8; a move rescales the row's O in tensor memory (moving it with every new maximum:
// window 190 -> 209 us, chunk 1470 -> 1580). Weights are rounded to the type (bf16 2^-8, fp16
// 2^-11 relative, one rounding a weight), and l is the fp32 sum of the rounded ones, so that a
// mean of equal values is that value and the roundings of a few large weights fall out. (The sum
// of unrounded ones: 64 prompts 69.1 -> 66.8 us, 32 cross prompts 95.7 -> 94.3, else under 1 %;
// of ones unpacked to fp32 first: 69.8 and 97.5.)
//
// Bound by the softmax warps: a tile of 64 x 256 scores takes 1700 cycles, of which the
// products need 900 (head_dim 128) and the exponentials 512 of their unit; the rest are the
// waits of two warps a scheduler that follow their scores step by step. Measured on GB300
// (us, in a graph): 2048 tokens behind 15953, 96 heads of 128, 1470 to 1510 (1150 TFLOP/s, 61 %
// of the library matrix product's burst rate and 68 % of its sustained one); 64 prompts of 150
// tokens, 32 heads on 8, 69; 4 chunks of 2000 tokens, windows of 1024, 16 heads of 256 on 8, 190.
// Tiles of 128 tokens with one S each, on an earlier build: 78 and 72 for the 64 prompts, 1555
// and 1540 for the chunk. The pairs of figures below are of one build each.
//
// Tiles arrive by TMA, one copy a block, from a 4-D view of the pool {64 elements, 8
// rows, head_dim / 64 chunks, 8-row groups}: a tile is then groups of swizzle atoms (8
// rows x 128 bytes) in equal strides, over tokens and over elements.
//
// Work: the items, in the order of the batch, are one list whose length counts the
// positions they see and kPromptStart for each item's start and end; every CTA takes an
// equal share, cut at whole tiles. Pieces of cut items go to the workspace in fp32 and a
// second kernel joins them by log-sum-exp, in the order of the tiles.
#pragma once

#include <cuda.h>

#include "device_common.cuh"
#include "even_split.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace pkv {

constexpr int kPromptSms = 152;    // CTAs: one per SM of a GB300
constexpr int kPromptTile = 64;    // tokens of a KV tile
// Tiles of a share where there is less work than SMs: every share more is one more piece to join. 5 tokens
// behind 4000, 8 heads on 1, take 34.3 us with one tile a share, 22.5 with two, 17.8 with three (heads of 256: 32.8,
// 23.8, 20.3); behind 1000, 8 heads on 2, 14.7, 13.0 and 13.5 (15.9, 13.7, 14.6); one token behind 500, 4 heads of 256
// on 1, 12.7, 11.2 and 12.4; a prompt of 300 there 20.0, 20.6 and 19.1.
constexpr int kPromptShareTiles = 2;
// What an item costs besides its positions, in positions: 64 prompts of 150 tokens take 92 us with
// 16, 69 with 128, 72 with 384.
constexpr int kPromptStart = 128;
// Cuts this near an item's end are moved there: the same prompts take 82 us with 64, 69 with 256 and
// 512; windows of 1024 196, 190 and 192.
constexpr int kPromptSnap = 256;
// A decode grid gives a single token one CTA a KV head, whose rate is near an SM's share of the memory's. One that
// would take kTailShares times as long as an even share of all single tokens is cut into pieces here instead. 60 tokens
// over 600 positions and one over 65000, 32 heads on 8: 991 us uncut, 95 cut, over 8000 143 and 58; 64 places with two
// tokens over 30000 469 and 66; behind a prefix 63 x 100 and one of 20000 329 and 66. Finding out costs tokens of equal
// lengths nothing measurable, and what follows prefixes 2 us.
constexpr int kTailShares = 2;
constexpr int kTailShort = 1024;  // (never worth that: 59 over 100 and one over 1000 26.9 us, over 1500 35.0 uncut and 29.7)
// The list is then made again, which takes as long as half a position a sequence: 3 long ones (up to 20000) among 16000
// short ones 363 us uncut and 336, among 65535 853 and 1319.
constexpr float kTailList = 0.5f;
constexpr int kTailAll = 0x7fffffff;
constexpr float kPromptLazy = 8.f;
// fp16 weights are 2^7 times as large, 2^(7 + 8) at most: one 2^-21 of the largest still has all its bits, and what
// fp16 loses of smaller ones is at most 2^-32 of the largest.
constexpr float kPromptHeadroom = 7.f;
constexpr int kPromptPieces = 4;   // pieces that the copying warp may be ahead
constexpr int kPromptNone = -1;
// A piece of one tile of rows goes to one warpgroup, the next to the other; from this many
// positions on, or with no piece behind it, to both. (256 and 4096 differ by less than 1 % in all cases
// but one: 8 sequences of 5 drafted tokens take 25.7 us with 256, 26.2 with 1024, 26.1 with 4096.)
constexpr int kPromptSplit = 1024;

template <int D>
struct PromptCfg {
  static constexpr int GROUPS = D == 256 ? 1 : 2;     // softmax warpgroups
  static constexpr int TILE = kPromptTile;
  static constexpr int CHUNKS = D / 64;
  static constexpr int SLOT = TILE * D * 2;           // bytes of a K or V tile
  static constexpr int SLOTS = D == 64 ? 16 : D == 128 ? 8 : 4;
  static constexpr int Q_TILE = 128 * D * 2;
  static constexpr int SOFTMAX = 128 * GROUPS;        // threads
  static constexpr int THREADS = SOFTMAX + 128;
  static constexpr int DEPTH = 2;                     // S buffers of a warpgroup
  static constexpr int STAGE = 2048;                  // bytes a softmax warp writes its output through
  static constexpr int STEP = CHUNKS * 1024;          // bytes of 8 tokens
  static constexpr int S_AT = GROUPS * D;             // columns of tensor memory: O, then two S
  static constexpr int COLUMNS = 512;
  static constexpr int LISTED = 384;                  // segments that are kept in shared memory
  static constexpr int STATS_AT = 1024, STAGE_AT = STATS_AT + 1024 * GROUPS, LIST_AT = STAGE_AT + STAGE * 4 * GROUPS;
  static constexpr int MISC = LIST_AT + LISTED * 32;
  static constexpr size_t SMEM_BYTES = 1024 + size_t(GROUPS) * Q_TILE + size_t(SLOTS) * SLOT + MISC;
  static_assert(S_AT + GROUPS * DEPTH * TILE <= COLUMNS, "tensor memory");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

// ---- the list of items ------------------------------------------------------
enum { kRowsCausal = 0, kRowsAll = 1, kRowsMembers = 2 };

// Queries that share a table: a sequence's; a group's members over their prefix
// (kRowsMembers); a member over the rest.
struct __align__(16) PromptSegment {
  int q0, nq;   // query tokens
  int table;    // sequence whose table holds the positions
  int lo, len;  // positions [lo, len)
  int kind;
  long long cost;  // of one head
};

__device__ __forceinline__ int prompt_clamp(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }
__device__ __forceinline__ int prompt_len(const PromptArgs& a, int s) {
  return prompt_clamp(a.context_lens[s], 0, a.max_blocks_per_seq * kBlock);
}
__device__ __forceinline__ int prompt_prefix(const PromptArgs& a, int group) {
  return prompt_clamp(a.prefix_blocks[group], 0, a.max_blocks_per_seq) * kBlock;
}
// The group of sequence s and the sequences it begins and ends with; -1: none.
__device__ __forceinline__ int prompt_group(const PromptArgs& a, int s, int* first, int* end) {
  if (a.num_groups == 0) return -1;
  int lo = 0, hi = a.num_groups - 1;  // the last group that starts at or before s
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.group_starts[mid] <= s) lo = mid;
    else hi = mid - 1;
  }
  *first = prompt_clamp(a.group_starts[lo], 0, a.num_seqs);
  *end = prompt_clamp(a.group_starts[lo + 1], *first, a.num_seqs);
  return s >= *first && s < *end ? lo : -1;
}
__device__ __forceinline__ PromptSegment prompt_segment(const PromptArgs& a, int i) {
  PromptSegment g;
  if (a.query_starts) {
    g.q0 = prompt_clamp(a.query_starts[i], 0, a.num_tokens);
    g.nq = prompt_clamp(a.query_starts[i + 1], g.q0, a.num_tokens) - g.q0;
    g.table = i;
    g.lo = 0;
    g.len = prompt_len(a, i);
    g.kind = a.causal ? kRowsCausal : kRowsAll;
  } else if (i < a.num_groups) {
    g.q0 = prompt_clamp(a.group_starts[i], 0, a.num_seqs);
    g.nq = prompt_clamp(a.group_starts[i + 1], g.q0, a.num_seqs) - g.q0;
    g.table = min(g.q0, a.num_seqs - 1);
    g.lo = 0;
    g.len = prompt_prefix(a, i);
    g.kind = kRowsMembers;
  } else {
    const int s = i - a.num_groups;
    int first, end;
    const int group = prompt_group(a, s, &first, &end);
    g.q0 = s;
    g.nq = 1;
    g.table = s;
    g.len = prompt_len(a, s);
    g.lo = group < 0 ? 0 : min(g.len, prompt_prefix(a, group));
    g.kind = kRowsAll;
  }
  return g;
}

// Whether the decode grid takes a segment: one query token of a sequence that sees up to `limit` positions.
__device__ __forceinline__ bool prompt_single(const PromptArgs& a, const PromptSegment& g, int limit) {
  if (!a.tails || g.kind == kRowsMembers || g.nq != 1) return false;
  return (a.window ? min(g.len - g.lo, a.window) : g.len - g.lo) <= limit;
}

// Positions [lo, hi) that block rb of T tokens of a segment sees, and the position of
// its first token (causal).
__device__ __forceinline__ void prompt_block(const PromptArgs& a, const PromptSegment& g, int rb, int T, int* lo, int* hi,
                                             int* base) {
  *lo = g.lo;
  *hi = g.len;
  *base = 0;
  if (g.kind == kRowsCausal) {
    *base = g.len - g.nq + rb * T;
    *hi = max(0, *base + min(T, g.nq - rb * T));
    *lo = a.window && *base >= a.window ? *base - a.window + 1 : 0;  // (any window up to 2^31 - 1, base < 0 too)
  }
}
// sum over i < n of max(0, x + i T), x > -2^32
__device__ __forceinline__ long long prompt_ramp(long long x, int T, int n) {
  const unsigned skip = x > 0 ? 0u : unsigned(-x) / unsigned(T) + 1u;
  if (skip >= unsigned(n)) return 0;
  const long long count = n - int(skip);
  return count * (x + (long long)skip * T) + T * (count * (count - 1) / 2);
}
// Cost of the first r blocks of one head of a segment.
__device__ __forceinline__ long long prompt_cost(const PromptArgs& a, const PromptSegment& g, int r, int T) {
  const long long start = (long long)kPromptStart * r;
  if (g.kind != kRowsCausal) return start + (long long)r * (g.len - g.lo);
  const int whole = min(r, g.nq / T);
  long long c = start + prompt_ramp((long long)g.len - g.nq + T, T, whole);
  if (r > whole) c += g.len;
  if (a.window) c -= prompt_ramp((long long)g.len - g.nq - a.window + 1, T, r);
  return c;
}

// A piece of an item, as every role of the CTA reads it. tiles < 0: no more.
struct PromptPiece {
  int q0, tokens;  // query tokens of the block
  int head;        // KV head
  int tiles;       // KV tiles of this piece
  int kv0;         // position of its first one
  int lo, hi;      // positions that some row sees
  int base;        // position of the first token (causal)
  int kind;
  int slot;        // of the workspace; kPromptNone: the item is whole
  int mode;
};
// Who takes a piece: one warpgroup; both, a tile of rows each; both, every other KV tile each.
enum { kPieceFirst = 0, kPieceSecond = 1, kPieceRows = 2, kPieceSplit = 3 };
// The KV tiles of a piece that warpgroup w takes: from `first` in steps of `step`.
struct PieceTiles {
  int first, step;
  bool any;
  __device__ __forceinline__ PieceTiles(int mode, int tiles, int w)
      : first(mode == kPieceSplit ? w : 0), step(mode == kPieceSplit ? 2 : 1),
        any(mode == w || (mode >= kPieceRows && (mode == kPieceRows || w < tiles))) {}
  __device__ __forceinline__ bool has(int t) const { return any && (step == 1 || (t & 1) == first); }
};

struct PromptShared {
  uint64_t slot_full[16], slot_empty[16];
  uint64_t q_full[2], q_empty[2], s_full[4], p_full[4], pv_done[4], join;
  uint64_t piece_full[kPromptPieces], piece_empty[kPromptPieces];
  uint64_t drain[2];  // after a wait gave up
  PromptPiece piece[kPromptPieces];
  long long scan[3];
  float sums[4];
  int most[4];
  long long first_base;
  int first_seg, limit;
  uint32_t tmem;
  int stop;    // a wait gave up: every role leaves
  int lock;    // a warp issues its MMAs
  // Tiles of each warpgroup in turn: K's slot of the ring (V's is the next) + 32 x phase + 64 x
  // (first of its piece) + 128 x (last) + 256 x (the other warpgroup uses it too); -1: no more.
  int tile[2][16];
  int copies[2];  // K and V copies issued for these
};
enum { kTilePhase = 32, kTileFirst = 64, kTileLast = 128, kTileShared = 256 };
static_assert(sizeof(PromptShared) <= 1024, "shared state");

// ---- tcgen05 ----------------------------------------------------------------
// D += A B with A (16-bit, two values a column) in tensor memory.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// 32 lanes (one a thread) x 32 columns.
__device__ __forceinline__ void tc_ld_32x32(uint32_t addr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(addr));
}
// 32 lanes (one a thread) x 16 columns.
__device__ __forceinline__ void tc_ld_32x16(uint32_t addr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(addr));
}
__device__ __forceinline__ void tc_st_32x16(uint32_t addr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(addr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
__device__ __forceinline__ int lds_acquire(uint32_t addr) {
  int v;
  asm volatile("ld.acquire.cta.shared.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts_release(uint32_t addr, int v) {
  asm volatile("st.release.cta.shared.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
__device__ __forceinline__ void st_global_if(bool on, void* p, const uint4& u) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t@p st.global.v4.b32 [%1], {%2, %3, %4, %5};\n\t}" ::"r"(
                   uint32_t(on)),
               "l"(p), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w)
               : "memory");
}
// Two fp32 operations an instruction.
__device__ __forceinline__ unsigned long long pair(float x, float y) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(unsigned long long p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long x, unsigned long long y, unsigned long long z) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
// x + and y + the values of a packed pair, in fp32.
template <typename T>
__device__ __forceinline__ void add_rounded(float& x, float& y, uint32_t w) {
  if (std::is_same<T, __half>::value)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.rn.f32.f16 %0, l, %0;\n\tadd.rn.f32.f16 %1, h, %1;\n\t}"
        : "+f"(x), "+f"(y)
        : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;\n\t}"
        : "+f"(x), "+f"(y)
        : "r"(w));
}
// Values that an asynchronous load wrote are used behind its wait only.
template <int N>
__device__ __forceinline__ void tc_loaded(float (&x)[N]) {
  tc_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(x[i]));
}

// Waits of a warp, all lanes: false when the limit ran out or another role gave up. The clock
// is looked at once in 64 tries only: reading it takes longer than most waits.
__device__ __forceinline__ bool prompt_wait(uint32_t bar, uint32_t parity, volatile int* stop, unsigned int* status) {
  unsigned long long t0 = 0;
  for (int tries = 0;; ++tries) {
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    if ((tries & 63) != 63) continue;
    const unsigned long long now = global_timer_ns();
    if (tries == 63) t0 = now;
    bool over = now - t0 > kWaitLimitNs;
    if (over && !*stop) {
      *stop = 1;
      flag(status, PKV_DEV_WAIT_TIMEOUT);
    }
    over = *stop;
    if (__any_sync(kFull, over)) return false;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(PromptCfg<D>::THREADS, 1)
prompt_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap q1_map,
              const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  using C = PromptCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem) + 1023) & ~uintptr_t(1023));
  unsigned char* q_mem = base;                              // per tile of rows: chunks of [128][64]
  unsigned char* ring = q_mem + C::GROUPS * C::Q_TILE;      // K and V tiles in turn
  PromptShared& sh = *reinterpret_cast<PromptShared*>(ring + C::SLOTS * C::SLOT);
  unsigned char* const misc = ring + C::SLOTS * C::SLOT;
  float2* const stats = reinterpret_cast<float2*>(misc + C::STATS_AT);            // [GROUPS][128] of a join
  unsigned char* const stage = misc + C::STAGE_AT;                                // per softmax warp
  PromptSegment* const list = reinterpret_cast<PromptSegment*>(misc + C::LIST_AT);  // the segments, where there are few,
  long long* const runs = reinterpret_cast<long long*>(list);                       // else the costs of the 96 runs of them
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int WARP_KV = C::SOFTMAX / 32, WARP_Q = WARP_KV + 1, WARP_MMA = WARP_KV + 2;

  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(smem_addr(&sh.slot_full[i]), 1);
      mbar_init(smem_addr(&sh.slot_empty[i]), 2);
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.q_full[i]), 1);
      mbar_init(smem_addr(&sh.q_empty[i]), 1);
    }
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_addr(&sh.s_full[i]), 1);
      mbar_init(smem_addr(&sh.p_full[i]), 128);
      mbar_init(smem_addr(&sh.pv_done[i]), 1);
    }
    mbar_init(smem_addr(&sh.join), C::SOFTMAX);
#pragma unroll 1
    for (int i = 0; i < kPromptPieces; ++i) {
      mbar_init(smem_addr(&sh.piece_full[i]), 1);
      mbar_init(smem_addr(&sh.piece_empty[i]), C::SOFTMAX / 32 + 1);
    }
    mbar_init_fence();
    sh.stop = 0;
    sh.copies[0] = sh.copies[1] = sh.lock = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&q_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&q1_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&k_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&v_map) : "memory");
  }
  if (warp == WARP_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                 "r"(uint32_t(C::COLUMNS))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  asm volatile("griddepcontrol.launch_dependents;");
  const bool scanner = warp >= C::SOFTMAX / 32 && warp != WARP_Q;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // The list: each thread of three warps sums a run of segments, a scan of the sums gives
  // every run's place, and the thread whose run holds this CTA's share's begin finds its segment.
  const int TQ = a.tile_tokens, TB = TQ * C::GROUPS;  // tokens of a tile of rows, and of a block
  const int cta = int(blockIdx.x), ctas = int(gridDim.x);
  long long begin = 0, end = 0, total = 0, quotient = 0;
  // The decode grid takes single tokens of up to `limit` positions: all, until it is known that some are too long.
  int limit = kTailAll, segs = a.num_groups + (a.tails && !a.query_starts ? 0 : a.num_seqs);
  auto segment = [&](int i) {
    PromptSegment g = prompt_segment(a, i);
    if (prompt_single(a, g, limit)) g.nq = 0;
    g.cost = g.nq ? prompt_cost(a, g, (g.nq + TB - 1) / TB, TB) : 0;
    return g;
  };
  if (a.tails && warp < 4) {
    // meanwhile softmax warps sum what single tokens see, and one of them works out the limit
    float sum = 0.f;  // (fp32 is near enough for a limit)
    int most = 0;
#pragma unroll 1
    for (int s = tid; s < a.num_seqs; s += 128) {
      int n = prompt_len(a, s);
      if (a.window) n = min(n, a.window);
      if (a.query_starts) {
        const int q0 = prompt_clamp(a.query_starts[s], 0, a.num_tokens);
        if (prompt_clamp(a.query_starts[s + 1], q0, a.num_tokens) - q0 != 1) n = 0;
      } else {
        int first, last;
        const int group = prompt_group(a, s, &first, &last);
        if (group >= 0) n -= min(n, prompt_prefix(a, group));
      }
      sum += float(n);
      most = max(most, n);
    }
    most = __reduce_max_sync(kFull, most);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == 0) {
      sh.sums[warp] = sum;
      sh.most[warp] = most;
    }
    asm volatile("bar.sync 2, 128;" ::: "memory");
    if (warp == 0) {
      const float even = (sh.sums[0] + sh.sums[1] + sh.sums[2] + sh.sums[3]) * (float(a.num_kv_heads) / kPromptSms);
      const float least = fmaxf(fmaxf(kTailShort, float(a.num_seqs) * kTailList), kTailShares * even);
      const int top = max(max(sh.most[0], sh.most[1]), max(sh.most[2], sh.most[3]));
      if (lane == 0) {
        sh.limit = float(top) <= least ? kTailAll : int(least);
        if (cta == 0) *a.limit = sh.limit;
      }
      asm volatile("bar.arrive 1, 128;" ::: "memory");
    }
  }
  if (scanner) {
    const int part = warp == WARP_KV ? 0 : warp - WARP_MMA + 1, runner = part * 32 + lane;
    int run0, run1;
    bool listed;
    long long at, mine;
    for (bool again = false;;) {
      const int per = (segs + 95) / 96;
      run0 = min(segs, runner * per);
      run1 = min(segs, run0 + per);
      listed = segs <= C::LISTED;
      mine = 0;
#pragma unroll 1
      for (int i = run0; i < run1; ++i) {
        const PromptSegment g = segment(i);
        mine += g.cost * a.num_kv_heads;
        if (listed) list[i] = g;
        if (cta == 0) {
          const int s = i - a.num_groups;
          if (s >= 0 && (a.context_lens[s] < 0 || a.context_lens[s] > a.max_blocks_per_seq * kBlock))
            flag(a.status, PKV_DEV_BAD_CONTEXT_LEN);
          const int32_t* starts = a.query_starts ? a.query_starts : i < a.num_groups ? a.group_starts : nullptr;
          if (starts && (starts[i] < 0 || starts[i + 1] < starts[i] || starts[i + 1] > a.num_tokens))
            flag(a.status, PKV_DEV_BAD_START);
        }
      }
      at = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(kFull, at, o);
        if (lane >= o) at += x;
      }
      if (lane == 31) sh.scan[part] = at;
      if (!listed) runs[runner] = mine;
      asm volatile("bar.sync 1, %0;" ::"r"(a.tails && !again ? 128 : 96) : "memory");
      if (!a.tails || again) break;
      again = true;
      limit = sh.limit;
      if (limit == kTailAll) break;
      segs = a.num_groups + a.num_seqs;
    }
    const long long s0 = sh.scan[0], s1 = sh.scan[1];
    total = s0 + s1 + sh.scan[2];
    at += (part > 0 ? s0 : 0) + (part > 1 ? s1 : 0) - mine;
    quotient = total >> 32 ? total / ctas : (long long)(unsigned(total) / unsigned(ctas));
    const EvenSplit split(total, ctas, quotient);
    begin = split.begin(cta);
    end = split.begin(cta + 1);
    if (begin < end && begin >= at && begin < at + mine) {
      int i = run0;
#pragma unroll 1
      for (; i + 1 < run1; ++i) {
        const long long c = listed ? list[i].cost : segment(i).cost;
        if (at + c * a.num_kv_heads > begin) break;
        at += c * a.num_kv_heads;
      }
      sh.first_seg = i;
      sh.first_base = at;
    }
    asm volatile("bar.sync 1, 96;" ::: "memory");
  }
  volatile int* stop = &sh.stop;
  auto wait = [&](uint64_t& bar, int phase) { return prompt_wait(smem_addr(&bar), uint32_t(phase) & 1, stop, a.status); };
  auto test = [&](uint64_t& bar, int phase) { return bool(__all_sync(kFull, mbar_test(smem_addr(&bar), uint32_t(phase) & 1))); };
  if (warp == WARP_KV) {
    // ---- pieces, and the copies of K and V ----
    const EvenSplit split(total, ctas, quotient);
    const bool listed = segs <= C::LISTED;
    const int snap = int(min((long long)kPromptSnap, quotient / 16));
    // generator of pieces
    int seg = sh.first_seg, cached = -64, h = 0, rb = 0, blocks = 0;
    long long seg_base = sh.first_base, item = 0;
    PromptSegment g{}, mine_g{};
    bool open = false;     // g, h, rb, item name the next item
    bool links = false, continued = false;  // what is written to desc
    auto cut = [&](long long at, int tiles) {  // tiles of an item before position `at` of its cost
      long long t = at <= kPromptStart ? 0 : (at - kPromptStart + C::TILE / 2) / C::TILE;
      if (t * C::TILE < snap) t = 0;
      if ((tiles - t) * C::TILE < snap || t > tiles) t = tiles;
      return int(t);
    };
    // The longest of n <= 256 members: what of their prefix lies behind it none of them sees, so that it is
    // neither read nor multiplied. (The list counts whole prefixes; its cuts are moved to the tiles there are.)
    auto longest = [&](int q0, int n) {
      int top = 0;
#pragma unroll
      for (int j = 0; j < 256; j += 32)
        if (j + lane < n) top = max(top, prompt_len(a, q0 + j + lane));
      return __reduce_max_sync(kFull, top);
    };
    int table = 0;  // of the piece generated last
    auto generate = [&](PromptPiece& p) {
      for (;;) {
        if (!open) {
          if (begin >= end || seg >= segs || seg_base >= end) {
            p.tiles = -1;
            return;
          }
          if (listed) {
            g = list[seg];
          } else {
            if (seg - cached >= 32) {  // the next 32 segments, one a lane
              cached = seg;
              if (seg + lane < segs) mine_g = segment(seg + lane);
            }
            // (what the grid takes is passed over, 32 at a time or a run: 4000 tokens of which 3 are cut 561 us without)
            const uint32_t rest = __ballot_sync(kFull, cached + lane < segs && mine_g.nq > 0) >> (seg - cached);
            if (rest == 0) {
              const int per = (segs + 95) / 96;
              for (seg = cached + 32; seg < segs && runs[seg / per] == 0;) seg = (seg / per + 1) * per;
              continue;
            }
            seg += __ffs(rest) - 1;
            const int src = seg - cached;
            g.q0 = __shfl_sync(kFull, mine_g.q0, src);
            g.nq = __shfl_sync(kFull, mine_g.nq, src);
            g.table = __shfl_sync(kFull, mine_g.table, src);
            g.lo = __shfl_sync(kFull, mine_g.lo, src);
            g.len = __shfl_sync(kFull, mine_g.len, src);
            g.kind = __shfl_sync(kFull, mine_g.kind, src);
            g.cost = __shfl_sync(kFull, mine_g.cost, src);
          }
          ++seg;
          if (g.nq == 0) continue;
          blocks = (g.nq + TB - 1) / TB;
          h = rb = 0;
          item = seg_base;
          if (begin > seg_base) {  // the share begins inside
            h = min(a.num_kv_heads - 1, int(float(begin - seg_base) / float(g.cost)));
            while (h > 0 && h * g.cost > begin - seg_base) --h;  // (but for the quotient's rounding)
            while (h + 1 < a.num_kv_heads && (h + 1) * g.cost <= begin - seg_base) ++h;
            item += h * g.cost;
            const long long rest = begin - item;
            long long before = 0;
            int top = blocks - 1;
#pragma unroll 1
            while (rb < top) {
              const int mid = (rb + top + 1) >> 1;
              const long long c = prompt_cost(a, g, mid, TB);
              if (c <= rest) {
                rb = mid;
                before = c;
              } else {
                top = mid - 1;
              }
            }
            item += before;
          }
          seg_base += g.cost * a.num_kv_heads;
          open = true;
        }
        if (item >= end) {
          p.tiles = -1;
          return;
        }
        prompt_block(a, g, rb, TB, &p.lo, &p.hi, &p.base);
        const long long start = item, cost = kPromptStart + p.hi - p.lo;
        if (g.kind == kRowsMembers) p.hi = min(p.hi, longest(g.q0 + rb * TB, min(TB, g.nq - rb * TB)));
        const int first = p.lo & ~(kBlock - 1), tiles = p.hi > p.lo ? (p.hi - first + C::TILE - 1) / C::TILE : 0;
        p.q0 = g.q0 + rb * TB;
        p.tokens = min(TB, g.nq - rb * TB);
        p.head = h;
        p.kind = g.kind;
        table = g.table;
        const int t0 = begin <= start ? 0 : cut(begin - start, tiles), t1 = end >= start + cost ? tiles : cut(end - start, tiles);
        item += cost;
        if (++rb == blocks) {
          rb = 0;
          if (++h == a.num_kv_heads) open = false;
        }
        if (tiles ? t0 >= t1 : begin > start) continue;
        p.tiles = t1 - t0;
        p.kv0 = first + t0 * C::TILE;
        const bool whole = t1 - t0 == tiles;
        p.slot = whole ? kPromptNone : 2 * cta + (t0 == 0 ? 1 : 0);
        if (lane == 0) {
          // the shares that hold the rest: up to the one with the item's end
          int last = cta;
          if (!whole && t0 == 0) last = split.of(start + cost - 1);
          if (a.query_starts) {
            if (!whole && t0 == 0) {
              a.desc[cta] = make_int4(p.q0, p.tokens, p.head, last);
              links = true;
            }
          } else if (t0 == 0) {
            a.link[(size_t(p.kind == kRowsMembers ? 0 : 1) * a.num_seqs + p.q0) * a.num_kv_heads + p.head] =
                whole ? make_int2(-1, -1) : make_int2(cta, last);
          }
          if (t0 > 0) continued = true;
        }
        return;
      }
    };
    const int32_t* row = nullptr;
    int nb = 0;
    auto load_ids = [&](int from) {
      const int j = from + lane;
      return j < nb ? row[j] : a.num_blocks;  // (rows outside the tensor read as zeros)
    };
    auto checked = [&](int id, int j) {
      if (id >= 0 && (id < a.num_blocks || j >= nb)) return id;
      flag(a.status, PKV_DEV_BAD_BLOCK_ID);
      return 0;
    };
    PromptPiece p{}, next;
    bool ok = true;  // warp-uniform
    int n = 0;       // tiles (K or V) copied
    int given[2] = {0, 0};  // tiles that each warpgroup was given alone
    int told[2] = {0, 0};   // tiles that each was told of
    constexpr int B = C::TILE / kBlock;  // blocks of a tile
    int first_ids = 0;
    for (int count = -1; ok && p.tiles >= 0; ++count) {
      if (count >= 0) {
        if (count >= kPromptPieces) ok = wait(sh.piece_empty[count % kPromptPieces], count / kPromptPieces - 1);
        if (!ok) break;
        const bool more = open ? item < end : seg < segs && seg_base < end;
        if (C::GROUPS == 1) p.mode = kPieceFirst;
        else if (p.tokens > TQ) p.mode = kPieceRows;
        else if (p.tiles * C::TILE >= kPromptSplit || (p.tiles > 1 && !more)) p.mode = kPieceSplit;
        else p.mode = given[1] < given[0] ? kPieceSecond : kPieceFirst;
        if (p.mode == kPieceFirst) given[0] += p.tiles + 1;
        if (p.mode == kPieceSecond) given[1] += p.tiles + 1;
        if (lane == 0) {
          sh.piece[count % kPromptPieces] = p;
          mbar_arrive(smem_addr(&sh.piece_full[count % kPromptPieces]));
        }
      }
      int from = p.kv0 / kBlock, ids = checked(first_ids, from + lane), ahead = p.tiles > 32 / B ? load_ids(from + 32) : 0;
      const int32_t* next_row = nullptr;
      int next_nb = 0, next_ids = 0;
#pragma unroll 1
      for (int t = 0; t < max(1, p.tiles); ++t) {
        if (t < p.tiles) {
          const int block = p.kv0 / kBlock + t * B;
          if (block >= from + 32) {
            from += 32;
            ids = checked(ahead, from + lane);
            ahead = load_ids(from + 32);
          }
          int z[B];
#pragma unroll
          for (int j = 0; j < B; ++j) z[j] = 2 * (__shfl_sync(kFull, ids, block - from + j) * a.num_kv_heads + p.head);
          const PieceTiles one(p.mode, p.tiles, 0), two(p.mode, p.tiles, 1);
          const bool uses[2] = {one.has(t), two.has(t)};
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const int slot = n % C::SLOTS;
            if (n >= C::SLOTS) ok = wait(sh.slot_empty[slot], n / C::SLOTS - 1);
            if (!ok) break;
            if (elect_one()) {
              const uint32_t bar = smem_addr(&sh.slot_full[slot]), dst = smem_addr(ring) + slot * C::SLOT;
              mbar_arrive_expect_tx(bar, C::SLOT);
#pragma unroll
              for (int j = 0; j < B; ++j) tma_load_4d(dst + j * 2 * C::STEP, kv ? &v_map : &k_map, 0, 0, 0, z[j], bar);
#pragma unroll
              for (int w = 0; w < C::GROUPS; ++w) {
                if (!uses[w]) continue;
                if (kv == 0)
                  sh.tile[w][told[w] % 16] = slot + (n / C::SLOTS & 1 ? kTilePhase : 0) + (t == (w ? two : one).first ? kTileFirst : 0) +
                                             (t + (w ? two : one).step >= p.tiles ? kTileLast : 0) + (p.mode == kPieceRows ? kTileShared : 0);
                sts_release(smem_addr(&sh.copies[w]), 2 * told[w] + 1 + kv);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          told[0] += uses[0];
          told[1] += uses[1];
        }
        if (t == 0) {
          // the next piece, and its first block ids on their way, once the first copies are
          const int32_t* const this_row = row;
          const int this_nb = nb;
          generate(next);
          row = next_row = a.block_tables + size_t(table) * a.max_blocks_per_seq;
          nb = next_nb = (next.hi + kBlock - 1) / kBlock;
          if (next.tiles > 0) next_ids = load_ids(next.kv0 / kBlock);
          row = this_row;
          nb = this_nb;
        }
      }
      if (!ok) break;
      p = next;
      first_ids = next_ids;
      row = next_row;
      nb = next_nb;
      if (p.tiles < 0) {  // the end is announced
        ++count;
        if (count >= kPromptPieces) ok = wait(sh.piece_empty[count % kPromptPieces], count / kPromptPieces - 1);
        if (ok && lane == 0) {
          sh.piece[count % kPromptPieces] = p;
          mbar_arrive(smem_addr(&sh.piece_full[count % kPromptPieces]));
          for (int w = 0; w < C::GROUPS; ++w) {
            sh.tile[w][told[w] % 16] = -1;
            sts_release(smem_addr(&sh.copies[w]), 2 * told[w] + 1);
          }
        }
      }
    }
    if (lane == 0) {
      if (a.query_starts && !links) a.desc[cta] = make_int4(0, 0, 0, -1);
      a.more[cta] = continued;
    }
    if (*stop) {  // wait (bounded) for the copies in flight
      for (int i = 0; i < C::SLOTS; ++i)
        if (n > i) mbar_wait_bounded(smem_addr(&sh.slot_full[i]), uint32_t((n - 1 - i) / C::SLOTS) & 1, 10000000ull);
    }
  } else if (warp == WARP_Q) {
    // ---- copies of Q: a tile of rows for each warpgroup that takes the piece ----
    int loads[2] = {0, 0};
    bool ok = true;
    for (int count = 0; ok; ++count) {
      ok = wait(sh.piece_full[count % kPromptPieces], count / kPromptPieces);
      if (!ok) break;
      const PromptPiece p = sh.piece[count % kPromptPieces];
      if (p.tiles < 0) break;
      for (int w = 0; ok && w < C::GROUPS; ++w) {
        if (p.tiles == 0 || !PieceTiles(p.mode, p.tiles, w).any) continue;
        if (loads[w] > 0) ok = wait(sh.q_empty[w], loads[w] - 1);
        if (!ok) break;
        ++loads[w];
        if (elect_one()) {
          const int from = p.mode == kPieceRows ? w * TQ : 0, tokens = min(TQ, p.tokens - from);
          const uint32_t bar = smem_addr(&sh.q_full[w]), dst = smem_addr(q_mem) + w * C::Q_TILE;
          // (rows that no copy writes hold what they held: their scores are not used)
          if (tokens == 1) {
            mbar_arrive_expect_tx(bar, uint32_t(C::CHUNKS * a.group * 128));
            for (int c = 0; c < C::CHUNKS; ++c)
              tma_load_4d(dst + c * (128 * 128), &q1_map, 0, p.head * a.group, p.q0 + from, c, bar);
          } else {
            mbar_arrive_expect_tx(bar, uint32_t(C::CHUNKS * TQ * a.group * 128));
            for (int c = 0; c < C::CHUNKS; ++c)
              tma_load_4d(dst + c * (128 * 128), &q_map, 0, p.head * a.group, p.q0 + from, c, bar);
          }
        }
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(smem_addr(&sh.piece_empty[count % kPromptPieces]));
    }
    if (*stop)
      for (int w = 0; w < C::GROUPS; ++w)
        if (loads[w] > 0) mbar_wait_bounded(smem_addr(&sh.q_full[w]), uint32_t(loads[w] - 1) & 1, 10000000ull);
  } else if (warp >= WARP_MMA && warp < WARP_MMA + C::GROUPS) {
    // ---- MMA issue: a warp for each warpgroup ----
    // As soon as the weights are there O += P V, and S of a tile as soon as its K and a buffer
    // are. The two warps issue by turns (`lock`), so that while one warpgroup has its products
    // made the other makes weights: side by side both would wait for both (a long chunk 1670 us
    // without, 1470 with; documents 104 and 100; 2048 tokens behind 8000, 32 heads of 64, 240 and 234;
    // 32 cross prompts 97 and 96; short pieces are even). One lane issues, the
    // others keep step, so that all of it stays in uniform registers. The loop is short, without
    // waits of its own, and reads what the copying warp has worked out: every instruction between
    // two products is one that the tensor cores wait for.
    const int w = warp - WARP_MMA;
    constexpr uint32_t id_s = tc_idesc<T>(128, C::TILE, false), id_o = tc_idesc<T>(128, D, false) | (1u << 16);
    const uint64_t q_desc = tc_desc(smem_addr(q_mem) + w * C::Q_TILE, 16, 1024);
    const uint64_t k_desc = tc_desc(smem_addr(ring), 16, C::STEP), v_desc = tc_desc(smem_addr(ring), 1024, C::STEP);
    const uint32_t copies_at = smem_addr(&sh.copies[w]);
    int copies = 0, loads = 0;    // copies seen, Qs waited for
    int s = 0, o = 0;             // S and O issued
    int next = 0, v0 = 0, v1 = 0; // tile of the next S; of those whose O is to come, the older first
    bool known = false, scores = false, done = false;
    unsigned long long t0 = 0;
    auto reached = [&](uint64_t& bar, int phase, bool asleep) {
      const uint32_t at = smem_addr(&bar), parity = uint32_t(phase) & 1;
      return bool(__all_sync(kFull, asleep ? mbar_try_wait(at, parity) : mbar_test(at, parity)));
    };
    for (int polls = 0;; ++polls) {
      if (copies < 2 * s + 1 || copies < 2 * o + 2) copies = __shfl_sync(kFull, lds_acquire(copies_at), 0);
      if (!known && copies > 2 * s) {
        next = __shfl_sync(kFull, sh.tile[w][s % 16], 0);
        known = true;
        done = next < 0;
      }
      // (what is the only thing to wait for is waited for asleep: polling takes turns from the softmax warps)
      if (known && !done && !scores)
        scores = reached(sh.slot_full[next & 31], next / kTilePhase, s == o) && (!(next & kTileFirst) || reached(sh.q_full[w], loads, s == o));
      const int bo = w * C::DEPTH + o % C::DEPTH, bs = w * C::DEPTH + s % C::DEPTH;
      const bool outputs = s > o && copies >= 2 * o + 2 && reached(sh.p_full[bo], o / C::DEPTH, done || s - o == C::DEPTH) &&
                           test(sh.slot_full[(v0 & 31) + 1], v0 / kTilePhase);
      const bool more = scores && s - o - (outputs ? 1 : 0) < C::DEPTH;
      if (!outputs && !more) {
        if (done && s == o) break;
        if ((polls & 63) != 63) continue;
        const unsigned long long now = __shfl_sync(kFull, global_timer_ns(), 0);
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitLimitNs && lane == 0 && !*stop) {
          *stop = 1;
          flag(a.status, PKV_DEV_WAIT_TIMEOUT);
        }
        __syncwarp();
        if (__any_sync(kFull, *stop)) break;
        continue;
      }
      t0 = 0;
      tc_fence_after();
      if (elect_one()) {
        if (C::GROUPS == 2) {  // (what holds it only issues: a bounded number of tries is enough, and no turn is needed to be right)
          for (int tries = 0; tries < 4096 && atomicExch(&sh.lock, 1); ++tries) {}
        }
        if (outputs) {
          const uint32_t p = tmem + C::S_AT + bo * C::TILE, slot = (v0 & 31) + 1;
          const uint64_t d = v_desc + slot * (C::SLOT >> 4);
#pragma unroll 1
          for (int e = 0; e < C::TILE / 16; ++e)
            tc_mma_ts(tmem + w * D, p + 8 * e, d + e * (2 * C::STEP >> 4), id_o, !((v0 & kTileFirst) && e == 0));
          tc_commit(smem_addr(&sh.pv_done[bo]));
          tc_commit(smem_addr(&sh.slot_empty[slot]));
          if (!(v0 & kTileShared)) tc_commit(smem_addr(&sh.slot_empty[slot]));  // (for both)
        }
        if (more) {
          const uint32_t slot = next & 31, d = tmem + C::S_AT + bs * C::TILE;
          const uint64_t k = k_desc + slot * (C::SLOT >> 4);
#pragma unroll 1
          for (int c = 0; c < C::CHUNKS; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              tc_mma(d, q_desc + c * (128 * 128 >> 4) + 2 * e, k + c * (1024 >> 4) + 2 * e, id_s, c + e > 0);
          tc_commit(smem_addr(&sh.s_full[bs]));
          tc_commit(smem_addr(&sh.slot_empty[slot]));
          if (!(next & kTileShared)) tc_commit(smem_addr(&sh.slot_empty[slot]));
          if (next & kTileLast) tc_commit(smem_addr(&sh.q_empty[w]));
        }
        if (C::GROUPS == 2) atomicExch(&sh.lock, 0);
      }
      __syncwarp();
      if (outputs) {
        v0 = v1;
        ++o;
      }
      if (more) {
        (s == o ? v0 : v1) = next;
        if (next & kTileFirst) ++loads;
        known = scores = false;
        ++s;
      }
    }
    if (__any_sync(kFull, *stop) && elect_one()) {  // let the products in flight end before the tensor memory is freed
      const uint32_t bar = smem_addr(&sh.drain[w]);
      mbar_init(bar, 1);
      mbar_init_fence();
      tc_commit(bar);
      mbar_wait_bounded(bar, 0, 10000000ull);
    }
    __syncwarp();
  } else if (warp < C::SOFTMAX / 32) {
    // ---- softmax and output: a thread a row ----
    constexpr float kHeadroom = std::is_same<T, __half>::value ? kPromptHeadroom : 0.f;
    const int wg = warp >> 2, quarter = warp & 3, r = 32 * quarter + lane;
    const int tok = r / a.group, sub = r - tok * a.group;  // token of the tile, head of the group
    const uint32_t lanes = uint32_t(32 * quarter) << 16;
    // The score's factor is taken in on the way to the exponent; one that is not positive before
    // the maximum.
    const bool scaled = !(a.scale_log2 > 0.f);
    const float factor = scaled ? 1.f : a.scale_log2;
    int steps = 0, n0 = 0, joins = 0;  // tiles done; ring index of the piece's first tile; joins waited for
    // V's phase may be looked at only once its copy is issued, when the one before is over.
    auto copied = [&](int copies) {
      unsigned long long t0 = 0;
      for (int polls = 0; __any_sync(kFull, lds_acquire(smem_addr(&sh.copies[wg])) < copies); ++polls) {
        if ((polls & 63) != 63) continue;
        const unsigned long long now = __shfl_sync(kFull, global_timer_ns(), 0);
        if (polls == 63) t0 = now;
        if (__any_sync(kFull, *stop)) return false;
        if (now - t0 > kWaitLimitNs) {
          *stop = 1;
          if (lane == 0) flag(a.status, PKV_DEV_WAIT_TIMEOUT);
        }
        __syncwarp();
      }
      return true;
    };
    for (int count = 0;; ++count) {
      if (!wait(sh.piece_full[count % kPromptPieces], count / kPromptPieces)) break;
      const PromptPiece p = sh.piece[count % kPromptPieces];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.piece_empty[count % kPromptPieces]));
      if (p.tiles < 0) break;
      const PieceTiles share(p.mode, p.tiles, wg);
      n0 += 2 * p.tiles;
      if (!share.any) continue;
      const bool rows = p.mode == kPieceRows;
      const int token = tok + (rows ? wg * TQ : 0);
      const bool valid = tok < TQ && token < p.tokens;
      int rlo = 0, rhi = 0x7fffffff;  // positions that this row sees
      if (valid) {
        rlo = p.lo;
        rhi = p.hi;
        if (p.kind == kRowsCausal) {
          rhi = max(0, p.base + token + 1);
          rlo = a.window ? max(0, rhi - a.window) : 0;
        } else if (p.kind == kRowsMembers) {
          rhi = min(rhi, prompt_len(a, p.q0 + token));
        }
      }
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int i = share.first; i < p.tiles; i += share.step, ++steps) {
        const int b = wg * C::DEPTH + steps % C::DEPTH;
        ok = wait(sh.s_full[b], steps / C::DEPTH);
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_at = tmem + lanes + C::S_AT + b * C::TILE;
        const int c0 = p.kv0 + i * C::TILE;
        // Masked scores are written back first, in a loop of its own: few tiles need it.
        const bool mask = __any_sync(kFull, c0 + C::TILE > rhi || c0 < rlo) || scaled;
        if (mask) {
#pragma unroll 1
          for (int h = 0; h < C::TILE; h += 32) {
            float x[32];
            tc_ld_32x32(s_at + h, x);
            tc_loaded(x);
            const uint32_t seen = bits_below(rhi - c0 - h) & ~bits_below(rlo - c0 - h);
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c] = (seen >> c) & 1u ? x[c] * (scaled ? a.scale_log2 : 1.f) : -INFINITY;
            tc_st_32x16(s_at + h, reinterpret_cast<uint32_t*>(x));
            tc_st_32x16(s_at + h + 16, reinterpret_cast<uint32_t*>(x + 16));
          }
          tc_wait_st();
        }
        float x[C::TILE];
#pragma unroll
        for (int h = 0; h < C::TILE; h += 32) tc_ld_32x32(s_at + h, x + h);
        tc_loaded(x);
        float tops[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < C::TILE - 4; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) tops[e] = max3(tops[e], x[c + e], x[c + 4 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) tops[e] = fmaxf(tops[e], x[C::TILE - 4 + e]);
        float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
        top *= factor;
        // (rows of no query score what shared memory held before: they ask for no move, or the bits of others
        // would depend on it)
        if (__any_sync(kFull, valid && top > m + kPromptLazy)) {
          const float now = fmaxf(m, top), al = m == -INFINITY ? 0.f : fast_exp2(m - now);
          m = now;
          l *= al;
          if (i > share.first) {  // O's products so far come before its rescaling
            ok = wait(sh.pv_done[b ^ 1], (steps - 1) / C::DEPTH);
            if (!ok) break;
            tc_fence_after();
            const uint32_t o_at = tmem + lanes + wg * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              tc_ld_32x16(o_at + c, o);
              tc_loaded(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= al;
              tc_st_32x16(o_at + c, reinterpret_cast<uint32_t*>(o));
            }
          }
        }
        // Then the weights, which take half the columns of the scores.
        const float ref = kHeadroom - (m == -INFINITY ? 0.f : m);
        const unsigned long long ref2 = pair(ref, ref), factor2 = pair(factor, factor);
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < C::TILE; h += 32) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = unpair(fma2(pair(x[h + 2 * e], x[h + 2 * e + 1]), factor2, ref2));
            const float2 f = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            w[e] = pack2<T>(f.x, f.y);
            add_rounded<T>(sum[e & 1], sum[2 + (e & 1)], w[e]);
          }
          tc_st_32x16(s_at + h / 2, w);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (c0 < p.lo || c0 + C::TILE > p.hi) {
          // rows that no query sees hold whatever the block holds (NaN included): as values
          // they must be zeros
          const int n = n0 - 2 * (p.tiles - i) + 1, slot = n % C::SLOTS;
          ok = copied(2 * steps + 2) && wait(sh.slot_full[slot], n / C::SLOTS);
          if (!ok) break;
          const int low = max(0, p.lo - c0), high = prompt_clamp(p.hi - c0, 0, C::TILE), held = min(C::TILE, (high + kBlock - 1) / kBlock * kBlock);
          for (int e = tid & 127; e < (low + held - high) * (D / 8); e += 128) {
            const int at = e / (D / 8), v = e % (D / 8), token_row = at < low ? at : high + at - low;
            *reinterpret_cast<uint4*>(ring + slot * C::SLOT + token_row / 8 * C::STEP + v / 8 * 1024 + token_row % 8 * 128 +
                                      v % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(smem_addr(&sh.p_full[b]));
      }
      if (!ok) break;
      const bool joint = p.mode == kPieceSplit;  // (which has two tiles at least)
      if (p.tiles > 0) {
        const int last = steps - 1;
        if (!wait(sh.pv_done[wg * C::DEPTH + last % C::DEPTH], last / C::DEPTH)) break;
        tc_fence_after();
      }
      float mine_f = 1.f, other_f = 0.f;  // factors of this warpgroup's O and of the other's
      if (joint) {
        stats[wg * 128 + r] = make_float2(m, l);
        tc_fence_before();
        mbar_arrive(smem_addr(&sh.join));
        if (!wait(sh.join, joins++)) break;
        tc_fence_after();
        const float2 o = stats[(wg ^ 1) * 128 + r];
        const float now = fmaxf(m, o.x);
        mine_f = m == -INFINITY ? 0.f : fast_exp2(m - now);
        other_f = o.x == -INFINITY ? 0.f : fast_exp2(o.x - now);
        m = now;
        l = l * mine_f + o.y * other_f;
      }
      // columns: all of this warpgroup's O, or half of both
      const int col0 = joint ? wg * (D / 2) : 0, cols = joint ? D / 2 : D;
      const int hq = p.head * a.group + sub;
      const size_t out_row = size_t(p.q0 + token) * a.num_q_heads + hq;
      const bool direct = a.query_starts && p.slot == kPromptNone;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      size_t part_row = 0;  // row of the partial results
      if (!direct) {
        part_row = p.slot == kPromptNone
                       ? a.slot_rows * size_t(2) * ctas + size_t(p.kind == kRowsMembers ? 0 : 1) * a.num_seqs * a.num_q_heads + out_row
                       : size_t(p.slot) * a.slot_rows + (rows ? wg * 128 : 0) + r;
        if (valid && col0 == 0) a.part_ml[part_row] = make_float2(m - kHeadroom, l);  // (l and O are 2^kHeadroom times as large)
      }
      const uint32_t o_at = tmem + lanes;
      // Results go through shared memory, so that four lanes write 64 bytes of a row together:
      // 16-byte column q of row r lies at column (q + r / 2) % 4. This lane then writes column
      // lane % 4 of rows lane / 4 + 8 k.
      unsigned char* const mine_s = stage + warp * C::STAGE;
      int rows_at[4];
      T* dst_at[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        rows_at[k] = __shfl_sync(kFull, valid ? int(out_row) : -1, 8 * k + lane / 4);
        dst_at[k] = static_cast<T*>(a.out) + size_t(max(0, rows_at[k])) * D + 8 * (lane & 3);
      }
#pragma unroll 1
      for (int c = col0; c < col0 + cols; c += 32) {
        float o[32];
        if (p.tiles > 0) {
          tc_ld_32x32(o_at + wg * D + c, o);
          if (joint) {
            float q[32];
            tc_ld_32x32(o_at + (wg ^ 1) * D + c, q);
            tc_loaded(q);
            tc_loaded(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = o[e] * mine_f + q[e] * other_f;
          } else {
            tc_loaded(o);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (direct) {
          uint4 u[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float* x = o + 8 * k;
            u[k] = make_uint4(pack2<T>(x[0] * inv, x[1] * inv), pack2<T>(x[2] * inv, x[3] * inv),
                              pack2<T>(x[4] * inv, x[5] * inv), pack2<T>(x[6] * inv, x[7] * inv));
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(mine_s + lane * 64 + ((k + lane / 2) & 3) * 16) = u[k];
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int from = 8 * k + lane / 4;
            u[k] = *reinterpret_cast<const uint4*>(mine_s + from * 64 + (((lane & 3) + from / 2) & 3) * 16);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) st_global_if(rows_at[k] >= 0, dst_at[k] + c, u[k]);
        } else if (valid) {
          float* dst = a.part_o + part_row * D + c;
#pragma unroll
          for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(dst + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      tc_fence_before();
      if (joint) {  // both are read: the next piece may write them
        mbar_arrive(smem_addr(&sh.join));
        if (!wait(sh.join, joins++)) break;
        tc_fence_after();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(uint32_t(C::COLUMNS)));
  }
}

// ---- joining the pieces -----------------------------------------------------
// One row's pieces, a warp a row and lane l columns 4 l .. (and 128 on): first the
// (maximum, sum) pairs, a piece a lane, then out = sum w o / sum w l, w = 2^(m - max m).
template <typename T, int D>
struct PromptJoin {
  static constexpr int V = (D + 127) / 128;  // float4s of a lane
  float M = -INFINITY, den = 0.f;
  float4 num[V] = {};
  __device__ __forceinline__ void scale(float f) {
    den *= f;
#pragma unroll
    for (int v = 0; v < V; ++v) num[v].x *= f, num[v].y *= f, num[v].z *= f, num[v].w *= f;
  }
  // up to 32 pieces: lane i names the row of piece i (on: there is one)
  __device__ __forceinline__ void add(const PromptArgs& a, bool on, size_t row, int pieces, int lane) {
    const float2 ml = on ? __ldcg(a.part_ml + row) : make_float2(-INFINITY, 0.f);
    float now = fmaxf(M, ml.x);
#pragma unroll
    for (int o = 16; o; o >>= 1) now = fmaxf(now, __shfl_xor_sync(kFull, now, o));
    // (a query that holds NaN has sums of NaN behind a maximum of -inf: they are joined, so that it gets NaN)
    scale(M == -INFINITY ? 0.f : fast_exp2(M - now));
    M = now;
    const float w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - now);
    float add = w * ml.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) add += __shfl_xor_sync(kFull, add, o);
    den += add;
#pragma unroll 4
    for (int i = 0; i < pieces; ++i) {
      const float wi = __shfl_sync(kFull, w, i);
      const size_t at = __shfl_sync(kFull, (unsigned long long)row, i);
      if (wi == 0.f) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = 4 * lane + 128 * v;
        if (c >= D) continue;
        const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D + c));
        num[v].x = fmaf(wi, x.x, num[v].x);
        num[v].y = fmaf(wi, x.y, num[v].y);
        num[v].z = fmaf(wi, x.z, num[v].z);
        num[v].w = fmaf(wi, x.w, num[v].w);
      }
    }
  }
  // the pieces of a cut item: share `first` holds its start, the others up to `last` what `more` says
  __device__ __forceinline__ void chain(const PromptArgs& a, int first, int last, int row, int lane) {
    first = max(0, min(first, a.shares - 1));
    last = max(first, min(last, a.shares - 1));
#pragma unroll 1
    for (int c = first; c <= last; c += 32) {
      const int mine = c + lane;
      const bool on = mine <= last && (mine == first || __ldcg(a.more + mine));
      add(a, on, size_t(2 * mine + (mine == first ? 1 : 0)) * a.slot_rows + row, min(32, last - c + 1), lane);
    }
  }
  // a sequence's part behind its prefix: cut, or whole
  __device__ __forceinline__ void own(const PromptArgs& a, int s, int hq, int h, int sub, int lane) {
    const int2 at = __ldcg(a.link + h + (size_t(a.num_seqs) + s) * a.num_kv_heads);
    if (at.x >= 0)
      chain(a, at.x, at.y, sub, lane);
    else
      add(a, lane == 0, a.slot_rows * size_t(2) * a.shares + (size_t(a.num_seqs) + s) * a.num_q_heads + hq, 1, lane);
  }
  __device__ __forceinline__ void keep(const PromptArgs& a, size_t row, int lane) {
    if (lane == 0) a.part_ml[row] = make_float2(M, den);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 4 * lane + 128 * v;
      if (c < D) *reinterpret_cast<float4*>(a.part_o + row * D + c) = num[v];
    }
  }
  __device__ __forceinline__ void write(const PromptArgs& a, size_t row, int lane) {
    const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 4 * lane + 128 * v;
      if (c < D)
        *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * D + c) =
            make_uint2(pack2<T>(num[v].x * inv, num[v].y * inv), pack2<T>(num[v].z * inv, num[v].w * inv));
    }
  }
};

// Both kernels are resident while the last one still runs. (A trial run of their code meanwhile
// took one token of cross attention from 38 us to 46 and prefixes from 97.1 to 98.2, and gave nothing.)

// Items that are cut: the warps of CTAs (share, 0 ..) take the rows of the one that starts in
// the share and goes on past it.
template <typename T, int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = int(blockIdx.y) * 8 + warp, step = int(gridDim.y) * 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 d = __ldcg(a.desc + blockIdx.x);  // query token, tokens, KV head, last share
  if (d.w < 0) return;
#pragma unroll 1
  for (int i = first; i < d.y * a.group; i += step) {
    const int token = i / a.group, sub = i - token * a.group, tile = token / a.tile_tokens;
    PromptJoin<T, D> j;
    j.chain(a, int(blockIdx.x), d.w, tile * 128 + (token - tile * a.tile_tokens) * a.group + sub, lane);
    j.write(a, size_t(d.x + token) * a.num_q_heads + d.z * a.group + sub, lane);
  }
}

// A sequence behind a prefix that is too long for the decode grid: what is kept of its prefix and its own pieces.
template <typename T, int D>
__device__ __noinline__ void prefix_join_long(const PromptArgs& a, size_t kept, int s, int hq, int lane) {
  const int h = hq / a.group;
  PromptJoin<T, D> j;
  j.add(a, lane == 0, kept, 1, lane);
  j.own(a, s, hq, h, hq - h * a.group, lane);
  j.write(a, size_t(s) * a.num_q_heads + hq, lane);
}

// Decode behind a prefix: a warp a (sequence, query head), over the pieces of its group's
// prefix and its own; with TAIL, where a decode grid takes the rest, the prefix alone, kept in
// fp32 for the grid.
template <typename T, int D, bool TAIL>
__global__ void __launch_bounds__(256) prefix_join_kernel(const PromptArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= int64_t(a.num_seqs) * a.num_q_heads) return;
  const int s = int(row / a.num_q_heads), hq = int(row - int64_t(s) * a.num_q_heads), h = hq / a.group, sub = hq - h * a.group;
  const size_t whole = a.slot_rows * size_t(2) * a.shares;  // rows of items that are not cut: prefixes, then own parts
  asm volatile("griddepcontrol.wait;" ::: "memory");
  PromptJoin<T, D> j;
  const int limit = TAIL ? __ldcg(a.limit) : 0;
  int first, end;
  const int group = prompt_group(a, s, &first, &end);
  if (TAIL && hq == 0 && lane == 0) a.from[s] = group < 0 ? 0 : min(prompt_len(a, s), prompt_prefix(a, group));
  bool kept = false;  // as it is to be kept
  if (group >= 0) {
    const int token = (s - first) % a.block_tokens, tile = token / a.tile_tokens;
    const int2 at = __ldcg(a.link + h + size_t(s - token) * a.num_kv_heads);
    if (at.x >= 0)
      j.chain(a, at.x, at.y, tile * 128 + (token - tile * a.tile_tokens) * a.group + sub, lane);
    else if (TAIL)
      kept = true;
    else
      j.add(a, lane == 0, whole + size_t(row), 1, lane);
  }
  if (TAIL) {
    if (!kept) j.keep(a, whole + size_t(row), lane);
    if (limit == kTailAll) return;
    const int len = prompt_len(a, s);
    if ((group < 0 ? len : len - prompt_prefix(a, group)) > limit) prefix_join_long<T, D>(a, whole + size_t(row), s, hq, lane);
    return;
  }
  j.own(a, s, hq, h, sub, lane);
  j.write(a, size_t(row), lane);
}

}  // namespace pkv
