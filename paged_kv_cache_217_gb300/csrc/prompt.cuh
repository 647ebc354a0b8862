// Attention of many query rows over the paged cache on the 5th-generation tensor
// cores: prompts, chunks of prompts and drafted tokens (causal), cross attention, and
// the decode of groups that share a prefix.
//
// A row is a (query token, query head) pair; the G heads of a KV head lie together, so
// that the K and V of a head are read once for all of them:
//     S = Q K^T (fp32),  p = 2^(scale log2(e) S - m),  O += P V,  l += sum p,  out = O / l.
// One CTA (1 per SM) takes pieces of items. An item is a block of up to 256 rows of one
// KV head (128 with head_dim 256) and the positions that any of them sees; a piece is
// some of its tiles of 128 tokens (64).
//
// Warps: two softmax warpgroups (a thread a row of the tile), one warp each that copies
// K and V, copies Q, and issues the MMAs. Warpgroup w owns S_w and O_w in tensor memory
// (S 128 columns, O head_dim). A block of more than 128 rows gives each warpgroup a tile
// of rows and every K and V tile is used by both; a smaller one (few queries, decode)
// gives both the same rows and every other tile, joined at the end. With head_dim 256 O
// leaves room for one warpgroup, whose tiles alternate between two S.
//  * S_w = Q K^T: both operands in shared memory, K-major, 128-byte swizzle.
//  * P overwrites S_w as 16-bit values, and is the A operand from there; V is read
//    MN-major from the tile as it lies.
// While one warpgroup works on its scores the tensor cores run the other's products.
// The running maximum is a reference that moves only when a score exceeds it by 2^8; a
// move rescales the row's O in tensor memory. Weights are rounded to the type (bf16
// 2^-8, fp16 2^-11 relative, one rounding a weight), and l is the fp32 sum of the rounded
// ones, so that the error is that of a weighted mean.
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
#include "latent_decode.cuh"
#include "launch.h"

namespace pkv {

constexpr int kPromptSms = 152;    // CTAs: one per SM of a GB300
constexpr int kPromptStart = 128;  // what an item costs besides its positions, in positions
constexpr int kPromptSnap = 512;   // cuts this near an item's end are moved there
constexpr float kPromptLazy = 8.f;
constexpr float kPromptHeadroom = 7.f;  // fp16 weights are 2^7 times as large (see kLatentHeadroom)
constexpr int kPromptPieces = 4;   // pieces that the copying warp may be ahead
constexpr int kPromptNone = -1;

template <int D>
struct PromptCfg {
  static constexpr int GROUPS = D == 256 ? 1 : 2;     // softmax warpgroups
  static constexpr int TILE = D == 256 ? 64 : 128;    // tokens
  static constexpr int ROWS = 128 * GROUPS;           // of an item
  static constexpr int CHUNKS = D / 64;
  static constexpr int SLOT = TILE * D * 2;           // bytes of a K or V tile
  static constexpr int SLOTS = D == 64 ? 8 : 4;
  static constexpr int Q_TILE = 128 * D * 2;
  static constexpr int SOFTMAX = 128 * GROUPS;        // threads
  static constexpr int THREADS = SOFTMAX + 96;
  static constexpr int STEP = CHUNKS * 1024;          // bytes of 8 tokens
  static constexpr int S_AT = GROUPS * D;             // columns of tensor memory: O, then S
  static constexpr int COLUMNS = 512;
  static constexpr int MISC = 1024 + 1024 * GROUPS;
  static constexpr size_t SMEM_BYTES = 1024 + size_t(GROUPS) * Q_TILE + size_t(SLOTS) * SLOT + MISC;
  static_assert(S_AT + 2 * TILE <= COLUMNS, "tensor memory");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

// ---- the list of items ------------------------------------------------------
enum { kRowsCausal = 0, kRowsAll = 1, kRowsMembers = 2 };

// Queries that share a table: a sequence's; a group's members over their prefix
// (kRowsMembers); a member over the rest.
struct PromptSegment {
  int q0, nq;   // query tokens
  int table;    // sequence whose table holds the positions
  int lo, len;  // positions [lo, len)
  int kind;
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
    *lo = a.window ? max(0, *base - a.window + 1) : 0;
  }
}
// sum over i < n of max(0, x + i T)
__device__ __forceinline__ long long prompt_ramp(long long x, int T, int n) {
  const int skip = x > 0 ? 0 : int(min((long long)n, -x / T + 1));
  const long long count = n - skip;
  return count <= 0 ? 0 : count * (x + (long long)skip * T) + T * (count * (count - 1) / 2);
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
};

struct PromptShared {
  uint64_t slot_full[8], slot_empty[8];
  uint64_t q_full, q_empty, s_full[2], p_full[2], pv_done[2], join;
  uint64_t piece_full[kPromptPieces], piece_empty[kPromptPieces];
  uint64_t drain;  // after a wait gave up
  PromptPiece piece[kPromptPieces];
  long long scan[12];
  long long first_base;
  int first_seg;
  uint32_t tmem;
  int stop;  // a wait gave up: every role leaves
};
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
__device__ __forceinline__ void tc_st_32x32(uint32_t addr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
      "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
      "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
      : "memory");
}
// Values that an asynchronous load wrote are used behind its wait only.
template <int N>
__device__ __forceinline__ void tc_loaded(float (&x)[N]) {
  tc_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(x[i]));
}

template <typename T, int D>
__global__ void __launch_bounds__(PromptCfg<D>::THREADS, 1)
prompt_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
              const __grid_constant__ CUtensorMap v_map) {
  using C = PromptCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem) + 1023) & ~uintptr_t(1023));
  unsigned char* q_mem = base;                              // per tile of rows: chunks of [128][64]
  unsigned char* ring = q_mem + C::GROUPS * C::Q_TILE;      // K and V tiles in turn
  PromptShared& sh = *reinterpret_cast<PromptShared*>(ring + C::SLOTS * C::SLOT);
  float2* const stats = reinterpret_cast<float2*>(ring + C::SLOTS * C::SLOT + 1024);  // [GROUPS][128] of a join
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int WARP_KV = C::SOFTMAX / 32, WARP_Q = WARP_KV + 1, WARP_MMA = WARP_KV + 2;

  if (tid == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_addr(&sh.slot_full[i]), 1);
      mbar_init(smem_addr(&sh.slot_empty[i]), 1);
    }
    mbar_init(smem_addr(&sh.q_full), 1);
    mbar_init(smem_addr(&sh.q_empty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.s_full[i]), 1);
      mbar_init(smem_addr(&sh.p_full[i]), 128);
      mbar_init(smem_addr(&sh.pv_done[i]), 1);
    }
    mbar_init(smem_addr(&sh.join), C::SOFTMAX);
    for (int i = 0; i < kPromptPieces; ++i) {
      mbar_init(smem_addr(&sh.piece_full[i]), 1);
      mbar_init(smem_addr(&sh.piece_empty[i]), C::SOFTMAX / 32 + 2);
    }
    mbar_init_fence();
    sh.stop = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&q_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&k_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&v_map) : "memory");
  }
  if (warp == WARP_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                 "r"(uint32_t(C::COLUMNS))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // The list: each thread sums a run of segments, a scan of the sums gives every
  // run's place, and the thread whose run holds this CTA's share's begin finds its
  // segment.
  const int TQ = a.tile_tokens, TB = TQ * C::GROUPS;  // tokens of a tile of rows, and of a block
  const int segs = a.num_groups + a.num_seqs;
  const int per = (segs + C::THREADS - 1) / C::THREADS;
  const int run0 = min(segs, tid * per), run1 = min(segs, run0 + per);
  auto segment_cost = [&](const PromptSegment& g) {
    return g.nq ? prompt_cost(a, g, (g.nq + TB - 1) / TB, TB) * a.num_kv_heads : 0ll;
  };
  long long mine = 0;
  for (int i = run0; i < run1; ++i) {
    if (blockIdx.x == 0) {
      const int s = i - a.num_groups;
      if (s >= 0 && (a.context_lens[s] < 0 || a.context_lens[s] > a.max_blocks_per_seq * kBlock))
        flag(a.status, PKV_DEV_BAD_CONTEXT_LEN);
      const int32_t* starts = a.query_starts ? a.query_starts : i < a.num_groups ? a.group_starts : nullptr;
      if (starts && (starts[i] < 0 || starts[i + 1] < starts[i] || starts[i + 1] > a.num_tokens))
        flag(a.status, PKV_DEV_BAD_START);
    }
    mine += segment_cost(prompt_segment(a, i));
  }
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(kFull, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) sh.scan[warp] = upto;
  __syncthreads();
  long long before = upto - mine, total = 0;
#pragma unroll
  for (int i = 0; i < C::THREADS / 32; ++i) {
    if (i < warp) before += sh.scan[i];
    total += sh.scan[i];
  }
  const int cta = int(blockIdx.x), ctas = int(gridDim.x);
  const long long begin = total * cta / ctas, end = total * (cta + 1) / ctas;
  if (begin < end && begin >= before && begin < before + mine) {
    long long at = before;
    int i = run0;
    for (;; ++i) {
      const long long c = segment_cost(prompt_segment(a, i));
      if (at + c > begin) break;
      at += c;
    }
    sh.first_seg = i;
    sh.first_base = at;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* stop = &sh.stop;
  auto wait = [&](uint64_t& bar, int phase) { return latent_wait(smem_addr(&bar), uint32_t(phase) & 1, stop, a.status); };

  if (warp == WARP_KV) {
    // ---- pieces, and the copies of K and V ----
    const int snap = int(min((long long)kPromptSnap, total / ctas / 16));
    // generator of pieces
    int seg = sh.first_seg, cached = -64, h = 0, rb = 0, blocks = 0;
    long long seg_base = sh.first_base, item = 0, per_head = 0;
    PromptSegment g{}, mine_g{};
    bool open = false;     // g, h, rb, item name the next item
    bool links = false, continued = false;  // what is written to desc
    auto cut = [&](long long at, int tiles) {  // tiles of an item before position `at` of its cost
      long long t = at <= kPromptStart ? 0 : (at - kPromptStart + C::TILE / 2) / C::TILE;
      if (t * C::TILE < snap) t = 0;
      if ((tiles - t) * C::TILE < snap || t > tiles) t = tiles;
      return int(t);
    };
    int table = 0;  // of the piece generated last
    auto generate = [&](PromptPiece& p) {
      for (;;) {
        if (!open) {
          if (begin >= end || seg >= segs || seg_base >= end) {
            p.tiles = -1;
            return;
          }
          if (seg - cached >= 32) {  // the next 32 segments, one a lane
            cached = seg;
            if (seg + lane < segs) mine_g = prompt_segment(a, seg + lane);
          }
          const int src = seg - cached;
          g.q0 = __shfl_sync(kFull, mine_g.q0, src);
          g.nq = __shfl_sync(kFull, mine_g.nq, src);
          g.table = __shfl_sync(kFull, mine_g.table, src);
          g.lo = __shfl_sync(kFull, mine_g.lo, src);
          g.len = __shfl_sync(kFull, mine_g.len, src);
          g.kind = __shfl_sync(kFull, mine_g.kind, src);
          ++seg;
          if (g.nq == 0) continue;
          blocks = (g.nq + TB - 1) / TB;
          per_head = prompt_cost(a, g, blocks, TB);
          h = rb = 0;
          item = seg_base;
          if (begin > seg_base) {  // the share begins inside
            h = int((begin - seg_base) / per_head);
            const long long rest = begin - seg_base - h * per_head;
            int top = blocks - 1;
            while (rb < top) {
              const int mid = (rb + top + 1) >> 1;
              if (prompt_cost(a, g, mid, TB) <= rest) rb = mid;
              else top = mid - 1;
            }
            item = seg_base + h * per_head + prompt_cost(a, g, rb, TB);
          }
          seg_base += per_head * a.num_kv_heads;
          open = true;
        }
        if (item >= end) {
          p.tiles = -1;
          return;
        }
        prompt_block(a, g, rb, TB, &p.lo, &p.hi, &p.base);
        const long long start = item, cost = kPromptStart + p.hi - p.lo;
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
          if (!whole && t0 == 0) {
            last = int((start + cost - 1) * ctas / total);
            while (last + 1 < ctas && total * (last + 1) / ctas <= start + cost - 1) ++last;
            while (total * last / ctas > start + cost - 1) --last;
          }
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
    auto set_table = [&](const PromptPiece& p) {
      row = a.block_tables + size_t(table) * a.max_blocks_per_seq;
      nb = (p.hi + kBlock - 1) / kBlock;
    };
    PromptPiece p, next;
    bool ok = true;  // warp-uniform
    int n = 0;       // tiles (K or V) copied
    int count = 0;   // pieces
    generate(p);
    set_table(p);
    int first_ids = p.tiles > 0 ? load_ids(p.kv0 / kBlock) : 0;
    for (;;) {
      if (count >= kPromptPieces) ok = __all_sync(kFull, wait(sh.piece_empty[count % kPromptPieces], count / kPromptPieces - 1));
      if (!ok) break;
      if (lane == 0) {
        sh.piece[count % kPromptPieces] = p;
        mbar_arrive(smem_addr(&sh.piece_full[count % kPromptPieces]));
      }
      ++count;
      if (p.tiles < 0) break;
      // the next piece, and its first block ids on their way
      const int32_t* const this_row = row;
      const int this_nb = nb;
      generate(next);
      set_table(next);
      const int next_ids = next.tiles > 0 ? load_ids(next.kv0 / kBlock) : 0;
      const int32_t* const next_row = row;
      const int next_nb = nb;
      row = this_row;
      nb = this_nb;
      constexpr int B = C::TILE / kBlock;  // blocks of a tile
      int from = p.kv0 / kBlock, ids = checked(first_ids, from + lane), ahead = p.tiles > 32 / B ? load_ids(from + 32) : 0;
      for (int t = 0; ok && t < p.tiles; ++t) {
        const int block = p.kv0 / kBlock + t * B;
        if (block >= from + 32) {
          from += 32;
          ids = checked(ahead, from + lane);
          ahead = load_ids(from + 32);
        }
        int z[B];
#pragma unroll
        for (int j = 0; j < B; ++j) z[j] = 2 * (__shfl_sync(kFull, ids, block - from + j) * a.num_kv_heads + p.head);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++n) {
          const int slot = n % C::SLOTS;
          if (n >= C::SLOTS) ok = ok && __all_sync(kFull, wait(sh.slot_empty[slot], n / C::SLOTS - 1));
          if (!ok) break;
          if (elect_one()) {
            const uint32_t bar = smem_addr(&sh.slot_full[slot]), dst = smem_addr(ring) + slot * C::SLOT;
            mbar_arrive_expect_tx(bar, C::SLOT);
#pragma unroll
            for (int j = 0; j < B; ++j) tma_load_4d(dst + j * 2 * C::STEP, kv ? &v_map : &k_map, 0, 0, 0, z[j], bar);
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      p = next;
      first_ids = next_ids;
      row = next_row;
      nb = next_nb;
    }
    if (lane == 0 && a.query_starts) {
      if (!links) a.desc[cta] = make_int4(0, 0, 0, -1);
      a.more[cta] = continued;
    } else if (lane == 0) {
      a.more[cta] = continued;
    }
    if (*stop) {  // wait (bounded) for the copies in flight
      for (int i = 0; i < C::SLOTS; ++i)
        if (n > i) mbar_wait_bounded(smem_addr(&sh.slot_full[i]), uint32_t((n - 1 - i) / C::SLOTS) & 1, 10000000ull);
    }
  } else if (warp == WARP_Q) {
    // ---- copies of Q ----
    int loads = 0;
    for (int count = 0;; ++count) {
      if (!__all_sync(kFull, wait(sh.piece_full[count % kPromptPieces], count / kPromptPieces))) break;
      const PromptPiece p = sh.piece[count % kPromptPieces];
      if (p.tiles < 0) break;
      if (p.tiles > 0) {
        if (loads > 0 && !__all_sync(kFull, wait(sh.q_empty, loads - 1))) break;
        ++loads;
        if (elect_one()) {
          const int tiles = p.tokens > TQ ? 2 : 1;
          mbar_arrive_expect_tx(smem_addr(&sh.q_full), uint32_t(tiles * C::CHUNKS * TQ * a.group * 128));
          for (int t = 0; t < tiles; ++t)
            for (int c = 0; c < C::CHUNKS; ++c)
              tma_load_4d(smem_addr(q_mem) + t * C::Q_TILE + c * (128 * 128), &q_map, 0, p.head * a.group, p.q0 + t * TQ, c,
                          smem_addr(&sh.q_full));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.piece_empty[count % kPromptPieces]));
    }
    if (*stop && loads > 0) mbar_wait_bounded(smem_addr(&sh.q_full), uint32_t(loads - 1) & 1, 10000000ull);
  } else if (warp == WARP_MMA) {
    // ---- MMA issue: one lane ----
    if (elect_one()) {
      constexpr uint32_t id_s = tc_idesc<T>(128, C::TILE, false), id_o = tc_idesc<T>(128, D, false) | (1u << 16);
      const uint64_t q_desc = tc_desc(smem_addr(q_mem), 16, 1024);
      const uint64_t k_desc = tc_desc(smem_addr(ring), 16, C::STEP), v_desc = tc_desc(smem_addr(ring), 1024, C::STEP);
      int n0 = 0, loads = 0, weights[2] = {0, 0};
      bool ok = true;
      for (int count = 0; ok; ++count) {
        ok = wait(sh.piece_full[count % kPromptPieces], count / kPromptPieces);
        if (!ok) break;
        const int tiles = sh.piece[count % kPromptPieces].tiles;
        const bool rows = C::GROUPS == 2 && sh.piece[count % kPromptPieces].tokens > TQ;  // two tiles of rows
        if (tiles < 0) break;
        mbar_arrive(smem_addr(&sh.piece_empty[count % kPromptPieces]));
        if (tiles == 0) continue;
        ok = wait(sh.q_full, loads++);
        const int steps = rows ? 2 * tiles : tiles;
        auto scores = [&](int j) {
          const int i = rows ? j >> 1 : j, half = rows ? j & 1 : 0, b = j & 1, n = n0 + 2 * i, slot = n % C::SLOTS;
          if (half == 0) ok = ok && wait(sh.slot_full[slot], n / C::SLOTS);
          if (!ok) return;
          tc_fence_after();
          const uint64_t q = q_desc + half * (C::Q_TILE >> 4), k = k_desc + slot * (C::SLOT >> 4);
#pragma unroll
          for (int c = 0; c < C::CHUNKS; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              tc_mma(tmem + C::S_AT + b * C::TILE, q + c * (128 * 128 >> 4) + 2 * e, k + c * (1024 >> 4) + 2 * e, id_s, c + e > 0);
          tc_commit(smem_addr(&sh.s_full[b]));
          if (!rows || half == 1) tc_commit(smem_addr(&sh.slot_empty[slot]));
          if (j == steps - 1) tc_commit(smem_addr(&sh.q_empty));
        };
        scores(0);
        if (ok && steps > 1) scores(1);
        for (int j = 0; ok && j < steps; ++j) {
          const int i = rows ? j >> 1 : j, half = rows ? j & 1 : 0, b = j & 1, n = n0 + 2 * i + 1, slot = n % C::SLOTS;
          ok = wait(sh.p_full[b], weights[b]++);
          if (half == 0) ok = ok && wait(sh.slot_full[slot], n / C::SLOTS);
          if (!ok) break;
          tc_fence_after();
          const uint32_t o = tmem + (C::GROUPS == 2 ? b * D : 0), w = tmem + C::S_AT + b * C::TILE;
          const bool fresh = C::GROUPS == 2 ? j < 2 : j == 0;
          const uint64_t v = v_desc + slot * (C::SLOT >> 4);
#pragma unroll
          for (int e = 0; e < C::TILE / 16; ++e) tc_mma_ts(o, w + 8 * e, v + e * (2 * C::STEP >> 4), id_o, !(fresh && e == 0));
          tc_commit(smem_addr(&sh.pv_done[b]));
          if (!rows || half == 1) tc_commit(smem_addr(&sh.slot_empty[slot]));
          if (j + 2 < steps) scores(j + 2);
        }
        n0 += 2 * tiles;
      }
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
    // ---- softmax and output: a thread a row ----
    constexpr float kHeadroom = std::is_same<T, __half>::value ? kPromptHeadroom : 0.f;
    const int wg = warp >> 2, quarter = warp & 3, r = 32 * quarter + lane;
    const int tok = r / a.group, sub = r - tok * a.group;  // token of the tile, head of the group
    const uint32_t lanes = uint32_t(32 * quarter) << 16;
    const uint32_t s_base = tmem + C::S_AT + lanes;
    int steps_done[2] = {0, 0};  // on each S (this warpgroup's, but for head_dim 256)
    int n0 = 0, joins = 0;
    for (int count = 0;; ++count) {
      if (!__all_sync(kFull, wait(sh.piece_full[count % kPromptPieces], count / kPromptPieces))) break;
      const PromptPiece p = sh.piece[count % kPromptPieces];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.piece_empty[count % kPromptPieces]));
      if (p.tiles < 0) break;
      const bool rows = C::GROUPS == 2 && p.tokens > TQ;
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
      // this warpgroup's KV tiles: all of them, or every other one
      const int stride = rows || C::GROUPS == 1 ? 1 : 2;
      bool ok = true;
      for (int i = rows || C::GROUPS == 1 ? 0 : wg; i < p.tiles; i += stride) {
        const int b = C::GROUPS == 2 ? wg : i & 1;
        ok = __all_sync(kFull, wait(sh.s_full[b], steps_done[b]));
        if (!ok) break;
        ++steps_done[b];
        tc_fence_after();
        const uint32_t s_at = s_base + b * C::TILE;
        float x[C::TILE];
#pragma unroll
        for (int c = 0; c < C::TILE; c += 32) tc_ld_32x32(s_at + c, x + c);
        tc_loaded(x);
        const int c0 = p.kv0 + i * C::TILE;
        float top = -INFINITY;
        if (__any_sync(kFull, c0 < rlo || c0 + C::TILE > rhi)) {
          const int from = rlo - c0, upto = rhi - c0;
#pragma unroll
          for (int c = 0; c < C::TILE; ++c) {
            x[c] = c >= from && c < upto ? x[c] * a.scale_log2 : -INFINITY;
            top = fmaxf(top, x[c]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < C::TILE; ++c) {
            x[c] *= a.scale_log2;
            top = fmaxf(top, x[c]);
          }
        }
        if (__any_sync(kFull, top > m + kPromptLazy)) {
          const float now = fmaxf(m, top), al = m == -INFINITY ? 0.f : fast_exp2(m - now);
          m = now;
          l *= al;
          if (i >= stride) {  // (all of this O's products so far are done: S came after them; but for head_dim 256)
            if (C::GROUPS == 1) ok = __all_sync(kFull, wait(sh.pv_done[b ^ 1], steps_done[b ^ 1] - 1));
            if (!ok) break;
            tc_fence_after();
            const uint32_t o_at = tmem + lanes + (C::GROUPS == 2 ? wg * D : 0);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tc_ld_32x32(o_at + c, o);
              tc_loaded(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= al;
              tc_st_32x32(o_at + c, reinterpret_cast<uint32_t*>(o));
            }
          }
        }
        const float ref = (m == -INFINITY ? 0.f : m) - kHeadroom;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < C::TILE; c += 64) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            w[e] = pack2<T>(fast_exp2(x[c + 2 * e] - ref), fast_exp2(x[c + 2 * e + 1] - ref));
            const float2 f = unpack2<T>(w[e]);
            sum[2 * (e & 1)] += f.x;
            sum[2 * (e & 1) + 1] += f.y;
          }
          tc_st_32x32(s_at + c / 2, w);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (c0 < p.lo || c0 + C::TILE > p.hi) {
          // rows that no query sees hold whatever the block holds (NaN included): as values
          // they must be zeros
          const int n = n0 + 2 * i + 1, slot = n % C::SLOTS;
          ok = __all_sync(kFull, wait(sh.slot_full[slot], n / C::SLOTS));
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
      const bool joint = C::GROUPS == 2 && !rows && p.tiles > 1;
      const bool idle = C::GROUPS == 2 && !rows && p.tiles <= 1 && wg == 1;  // nothing to do but to keep count
      n0 += 2 * p.tiles;
      if (idle) continue;
      if (p.tiles > 0) {
        const int b = C::GROUPS == 2 ? wg : (p.tiles - 1) & 1;
        if (!__all_sync(kFull, wait(sh.pv_done[b], steps_done[b] - 1))) break;
        tc_fence_after();
      }
      float mine_f = 1.f, other_f = 0.f;  // factors of this warpgroup's O and of the other's
      if (joint) {
        stats[wg * 128 + r] = make_float2(m, l);
        tc_fence_before();
        mbar_arrive(smem_addr(&sh.join));
        if (!__all_sync(kFull, wait(sh.join, joins++))) break;
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
        if (valid && col0 == 0) a.part_ml[part_row] = make_float2(m, l);
      }
      const uint32_t o_at = tmem + lanes;
#pragma unroll 1
      for (int c = col0; c < col0 + cols; c += 32) {
        float o[32];
        if (p.tiles > 0) {
          tc_ld_32x32(o_at + (C::GROUPS == 2 ? wg * D : 0) + c, o);
          tc_loaded(o);
          if (joint) {
            float q[32];
            tc_ld_32x32(o_at + (wg ^ 1) * D + c, q);
            tc_loaded(q);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = o[e] * mine_f + q[e] * other_f;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (!valid) continue;
        if (direct) {
          T* dst = static_cast<T*>(a.out) + out_row * D + c;
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 u;
            u.x = pack2<T>(o[e] * inv, o[e + 1] * inv);
            u.y = pack2<T>(o[e + 2] * inv, o[e + 3] * inv);
            u.z = pack2<T>(o[e + 4] * inv, o[e + 5] * inv);
            u.w = pack2<T>(o[e + 6] * inv, o[e + 7] * inv);
            if (l == 0.f) u = make_uint4(0u, 0u, 0u, 0u);  // (a row that sees nothing of what its tile holds)
            *reinterpret_cast<uint4*>(dst + e) = u;
          }
        } else {
          float* dst = a.part_o + part_row * D + c;
#pragma unroll
          for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(dst + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      tc_fence_before();
      if (joint) {  // both are read: the next piece may write them
        mbar_arrive(smem_addr(&sh.join));
        if (!__all_sync(kFull, wait(sh.join, joins++))) break;
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
    if (now == -INFINITY) return;
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
    for (int c = first; c <= last; c += 32) {
      const int mine = c + lane;
      const bool on = mine <= last && (mine == first || __ldcg(a.more + mine));
      add(a, on, size_t(2 * mine + (mine == first ? 1 : 0)) * a.slot_rows + row, min(32, last - c + 1), lane);
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

// Items that are cut: CTA (share, y) takes every gridDim.y-th eighth of the rows of the
// one that starts in the share and goes on past it.
template <typename T, int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 d = __ldcg(a.desc + blockIdx.x);  // query token, tokens, KV head, last share
  if (d.w < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = int(blockIdx.y) * 8 + warp; i < d.y * a.group; i += int(gridDim.y) * 8) {
    const int token = i / a.group, sub = i - token * a.group, tile = token / a.tile_tokens;
    PromptJoin<T, D> j;
    j.chain(a, int(blockIdx.x), d.w, tile * 128 + (token - tile * a.tile_tokens) * a.group + sub, lane);
    j.write(a, size_t(d.x + token) * a.num_q_heads + d.z * a.group + sub, lane);
  }
}

// Decode behind a prefix: a warp a (sequence, query head), over the pieces of its group's
// prefix and its own.
template <typename T, int D>
__global__ void __launch_bounds__(256) prefix_join_kernel(const PromptArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= int64_t(a.num_seqs) * a.num_q_heads) return;
  const int s = int(row / a.num_q_heads), hq = int(row - int64_t(s) * a.num_q_heads), h = hq / a.group, sub = hq - h * a.group;
  const size_t whole = a.slot_rows * size_t(2) * a.shares;  // rows of items that are not cut: prefixes, then own parts
  PromptJoin<T, D> j;
  auto item = [&](int kind, int q0, int slot_row) {
    const int2 link = __ldcg(a.link + (size_t(kind) * a.num_seqs + q0) * a.num_kv_heads + h);
    if (link.x < 0) j.add(a, lane == 0, whole + (size_t(kind) * a.num_seqs + s) * a.num_q_heads + hq, 1, lane);
    else j.chain(a, link.x, link.y, slot_row, lane);
  };
  int first, end;
  if (prompt_group(a, s, &first, &end) >= 0) {
    const int token = (s - first) % a.block_tokens, tile = token / a.tile_tokens;
    item(0, s - token, tile * 128 + (token - tile * a.tile_tokens) * a.group + sub);
  }
  item(1, s, sub);
  j.write(a, size_t(row), lane);
}

}  // namespace pkv
