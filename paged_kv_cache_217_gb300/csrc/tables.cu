// Block tables and slot maps on the device: what the host block manager does
// for a batch (append with copy-on-write, release), as kernels, so that a
// captured decode loop needs no host round trip ([S] "KV キャッシュマネージャ":
// tokens fill the last block, a new block is taken when it is full, blocks go
// back on finish; [S] "並列サンプリングやビームサーチでの共有": a shared block
// is copied when a write reaches it).
//
// pkv_extend_block_tables, with L = context_lens[s], n = new_tokens[s]:
//   cow_s   = n > 0, L % 16 != 0 and the last block still shared when s's turn
//             comes: of the batch's k-th earlier sequence with that last block
//             (each took a copy), refcount - k > 1
//   fresh_s = ceil((L + n) / 16) - ceil(L / 16)
//   first_s = sum over earlier sequences of cow + fresh (an exclusive scan)
//   the i-th block of s (its copy first, then its new blocks in order) is
//   free_stack[count - 1 - first_s - i]
// -- exactly the blocks that the host manager pops for the same appends in
// batch order. Two phases: one CTA scans the batch (phase 1: offsets into the
// workspace, and the all-or-nothing checks), then every table entry and slot
// is filled independently (phase 2), each warp finding its sequences in the
// offsets by 32 probes a round (a binary search per thread: 11.4 us against 10.3
// for 700 prompts of 1.2M tokens, at 4 slots a thread in CTAs of 256). Bound by launch latency for a decode step and
// by the slot map's 8 bytes a token for prompts. A batch of at most
// kFusedSeqs sequences and kFusedSlots slots runs both phases in one CTA, with
// the offsets in shared memory.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "device_common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kFusedSeqs = 1024;
constexpr int kFusedSlots = 4096;  // 4000 slots of 1000 sequences: 6.2 us, in two kernels 8.7; 16000: 13.5, 8.3
constexpr int kFillThreads = 128;
// Slots a thread takes at a time. One CTA: 1 while that is one turn (256 slots 4.4
// us; 4 a thread 5.7), else 4 (4000 slots 6.2; 1 a thread 8.9). A grid: 2 (300000
// slots 6.6 us; 4 7.0, 8 7.4), from kManySlots 4 (600000 slots 7.3; 2 8.2; 1.2M 9.6;
// 2 11.4, 8 9.6).
constexpr int kManySlots = 400000;

// Per-batch results of phase 1, in the workspace (or shared memory).
struct Scan {
  int32_t* len;    // [S] lengths before the call
  int32_t* tok;    // [S + 1] first new token of each sequence
  int32_t* blk;    // [S + 1] first taken block of each sequence
  int32_t* cow;    // [S] the block to copy from, or -1
  int32_t* pair;   // [S] index of the sequence's copy pair
  int32_t* last;   // [S] shared last block of a sequence that appends into it, or -1
  int32_t* head;   // {ok, free count, pairs, 0}
};

__host__ __device__ inline size_t scan_ints(int S) { return size_t(6) * S + 2 + 4; }

__device__ __forceinline__ Scan scan_of(int32_t* p, int S) {
  return Scan{p, p + S, p + 2 * S + 1, p + 3 * S + 2, p + 4 * S + 2, p + 5 * S + 2, p + 6 * S + 2};
}

// Exclusive scans of C values over the CTA; every thread calls it. total: the
// CTA's sums.
template <typename V, int C>
__device__ __forceinline__ void cta_exclusive(V (&v)[C], V (*warp_sum)[C], V (&total)[C]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V x[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    x[c] = v[c];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const V n = __shfl_up_sync(kFull, x[c], o);
      if (lane >= o) x[c] += n;
    }
  }
  __syncthreads();  // earlier readers of warp_sum are done
  if (lane == 31) {
#pragma unroll
    for (int c = 0; c < C; ++c) warp_sum[warp][c] = x[c];
  }
  __syncthreads();
  if (warp < C) {  // warp c scans value c of the warps' sums
    V w = warp_sum[lane][warp];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const V n = __shfl_up_sync(kFull, w, o);
      if (lane >= o) w += n;
    }
    warp_sum[lane][warp] = w;
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < C; ++c) {
    total[c] = warp_sum[kThreads / 32 - 1][c];
    v[c] = x[c] - v[c] + (warp ? warp_sum[warp - 1][c] : V(0));
  }
}

// Phase 1, one CTA of kThreads threads.
__device__ __forceinline__ void scan_batch(const ExtendArgs& a, const Scan& w) {
  __shared__ long long wsum[32][2];
  __shared__ unsigned int flags;
  const int S = a.num_seqs;
  const long long max_len = (long long)a.max_blocks * kBlock;
  if (threadIdx.x == 0) flags = 0u;
  __syncthreads();
  const int count = *a.free_count;
  unsigned int bad = count < 0 || count > a.num_blocks ? PKV_DEV_BAD_BLOCK_ID : 0u;
  bool sharing = false;
  int n = 0, L = 0, last = -1;  // (kept for a batch of one sequence a thread)
  for (int s = threadIdx.x; s < S; s += kThreads) {
    L = a.context_lens[s];
    n = a.new_tokens[s];
    const bool ok = L >= 0 && n >= 0 && (long long)L + n <= max_len;
    if (!ok) {
      bad |= PKV_DEV_BAD_CONTEXT_LEN;
      L = n = 0;  // the call fails
    }
    last = -1;
    if (a.refcounts && n > 0 && L % kBlock) {
      const int b = a.block_tables[size_t(s) * a.max_blocks + L / kBlock];
      if (b >= 0 && b < a.num_blocks && a.refcounts[b] > 1) last = b;  // a bad id is flagged where it is used
    }
    sharing |= last >= 0;
    w.len[s] = L;
    w.last[s] = last;
  }
  if (bad) atomicOr(&flags, bad);
  const bool any_sharing = __syncthreads_or(sharing);

  long long tok0 = 0, blk0 = 0, pair0 = 0;
  for (int base = 0; base < S; base += kThreads) {
    const int s = base + threadIdx.x;
    long long v[2] = {0, 0}, total[2];
    int cow = 0;
    if (s < S) {
      if (S > kThreads) {
        L = w.len[s];
        last = w.last[s];
        n = a.new_tokens[s];
        const long long raw = a.context_lens[s];
        if (raw < 0 || n < 0 || raw + n > max_len) n = 0;
      }
      if (any_sharing && last >= 0) {
        // (every earlier sequence of the batch: 256 forked ones 7.2 us against 3.8 for a
        // call without sharing, 1024 19, 4096 187, 65532 44 ms)
        int rank = 0;
        for (int e = 0; e < s; ++e) rank += w.last[e] == last ? 1 : 0;
        cow = a.refcounts[last] - rank > 1 ? 1 : 0;
      }
      v[0] = n;
      v[1] = (L + n + kBlock - 1) / kBlock - (L + kBlock - 1) / kBlock + cow;
    }
    cta_exclusive<long long, 2>(v, wsum, total);
    const long long t = tok0 + v[0], bl = blk0 + v[1];
    tok0 += total[0];
    blk0 += total[1];
    long long pr = pair0;
    if (any_sharing) {
      long long c[2] = {cow, 0}, all[2];
      cta_exclusive<long long, 2>(c, wsum, all);
      pr += c[0];
      pair0 += all[0];
    }
    if (s < S) {
      w.tok[s] = int(t < INT_MAX ? t : INT_MAX);
      w.blk[s] = int(bl < INT_MAX ? bl : INT_MAX);
      w.cow[s] = cow ? last : -1;
      w.pair[s] = int(pr);
    }
  }
  if (threadIdx.x == 0) {
    unsigned int f = flags;
    if (tok0 > a.num_slots) f |= PKV_DEV_BAD_SLOT;
    if (blk0 > count && !(f & PKV_DEV_BAD_BLOCK_ID)) f |= PKV_DEV_OUT_OF_BLOCKS;
    if (f) flag(a.status, f);
    const bool ok = f == 0u;
    w.tok[S] = ok ? int(tok0) : 0;
    w.blk[S] = ok ? int(blk0) : 0;
    w.head[0] = ok ? 1 : 0;
    w.head[1] = count;
    w.head[2] = ok ? int(pair0) : 0;
    w.head[3] = int(f);
  }
}

// The last s in [lo, hi) with off[s] <= i (off ascending, off[lo] <= i).
__device__ __forceinline__ int owner(const int32_t* off, int lo, int hi, int i) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// The same in [0, S) for one i of the whole warp, 32 probes a round.
__device__ __forceinline__ int warp_owner(const int32_t* off, int S, int i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = S;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const int c = __popc(__ballot_sync(kFull, at < n && off[lo + at] <= i)) - 1;
    lo += c * step;
    n = min(step, n - c * step);
  }
  return lo;
}

// The i-th block taken by the batch, or -1 (flagged) if the stack holds none.
__device__ __forceinline__ int taken(const ExtendArgs& a, int count, int i) {
  const int b = a.free_stack[count - 1 - i];
  if (b >= 0 && b < a.num_blocks) return b;
  flag(a.status, PKV_DEV_BAD_BLOCK_ID);
  return -1;
}

// Phase 2: thread `tid` of `threads`. WARP: the offsets are in global memory, so a
// warp searches them together (in shared memory each thread does).
// U: slots a thread takes at a time.
template <bool WARP, int U>
__device__ __forceinline__ void fill(const ExtendArgs& a, const Scan& w, int64_t tid, int64_t threads) {
  const int S = a.num_seqs;
  const bool ok = w.head[0] != 0;
  const int count = w.head[1], tokens = w.tok[S], blocks = w.blk[S];
  const int lane = threadIdx.x & 31;
  for (int64_t w0 = (tid - lane) * U; w0 < a.num_slots; w0 += threads * U) {
    const int64_t i0 = w0 + lane * U;
    int64_t slot[U];
    int s = 0;
    if (!WARP) {
      if (i0 < tokens) s = owner(w.tok, 0, S, int(i0));
    } else if (w0 < tokens) {  // the sequences of the warp's first and last token, then this thread's between them
      const int first = warp_owner(w.tok, S, int(w0));
      const int last = warp_owner(w.tok, S, int(min(w0 + 32 * U, int64_t(tokens)) - 1));
      s = owner(w.tok, first, last + 1, int(min(i0, int64_t(tokens) - 1)));
    }
    int begin = 0, end = 0, L = 0, blk = 0, copied = 0;  // of sequence s
    auto enter = [&]() {
      begin = w.tok[s];
      end = w.tok[s + 1];
      L = w.len[s];
      blk = w.blk[s];
      copied = w.cow[s] >= 0 ? 1 : 0;
    };
    if (i0 < tokens) enter();
    int at = -1, phys = -1;  // block index and id of the previous token
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u;
      slot[u] = -1;
      if (i >= tokens) continue;
      while (i >= end) {
        ++s;
        enter();
        at = -1;
      }
      const int pos = L + int(i - begin), j = pos / kBlock;
      if (j != at) {
        const int have = (L + kBlock - 1) / kBlock;
        at = j;
        if (j >= have) {
          phys = taken(a, count, blk + copied + j - have);
        } else if (copied) {
          phys = taken(a, count, blk);
        } else {
          phys = a.block_tables[size_t(s) * a.max_blocks + j];
          if (phys < 0 || phys >= a.num_blocks) {
            flag(a.status, PKV_DEV_BAD_BLOCK_ID);
            phys = -1;
          }
        }
      }
      if (phys >= 0) slot[u] = int64_t(phys) * kBlock + pos % kBlock;
    }
    if (U > 1 && i0 + U <= a.num_slots && a.slots_aligned) {
      longlong2* dst = reinterpret_cast<longlong2*>(a.slot_mapping + i0);
#pragma unroll
      for (int u = 0; u + 1 < U; u += 2) dst[u / 2] = make_longlong2(slot[u], slot[u + 1]);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u < a.num_slots) a.slot_mapping[i0 + u] = slot[u];
    }
  }
  for (int64_t w0 = tid - lane; w0 < blocks; w0 += threads) {
    const int64_t i = w0 + lane;
    int first = 0, last = S - 1;
    if (WARP) {
      first = warp_owner(w.blk, S, int(w0));
      last = warp_owner(w.blk, S, int(min(w0 + 32, int64_t(blocks)) - 1));
    }
    if (i >= blocks) continue;
    const int s = owner(w.blk, first, last + 1, int(i));
    const int k = int(i) - w.blk[s], src = w.cow[s], have = (w.len[s] + kBlock - 1) / kBlock;
    const int b = taken(a, count, int(i));
    const int j = src >= 0 ? have - 1 + k : have + k;
    a.block_tables[size_t(s) * a.max_blocks + j] = b;
    if (a.refcounts && b >= 0) a.refcounts[b] = 1;
    if (src >= 0 && k == 0) {
      atomicSub(a.refcounts + src, 1);
      a.cow_pairs[2 * size_t(w.pair[s])] = src;
      a.cow_pairs[2 * size_t(w.pair[s]) + 1] = b;
    }
  }
  for (int64_t s = tid; s < S; s += threads) {
    // (a failed call leaves the lengths as they were, valid or not)
    if (ok) a.new_lens[s] = w.len[s] + (w.tok[s + 1] - w.tok[s]);
    else if (a.new_lens != a.context_lens) a.new_lens[s] = a.context_lens[s];
    if (a.cow_pairs && s >= w.head[2]) a.cow_pairs[2 * s] = a.cow_pairs[2 * s + 1] = -1;
  }
  if (tid == 0) {
    *a.new_free_count = count - blocks;
    if (a.info) {
      a.info[0] = w.head[3];
      a.info[1] = tokens;
      a.info[2] = blocks;
      a.info[3] = w.head[2];
    }
  }
}

__global__ void __launch_bounds__(kThreads) scan_kernel(const ExtendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  scan_batch(a, scan_of(a.workspace, a.num_seqs));
}

template <int U>
__global__ void __launch_bounds__(kFillThreads) fill_kernel(const ExtendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  fill<true, U>(a, scan_of(a.workspace, a.num_seqs), int64_t(blockIdx.x) * blockDim.x + threadIdx.x,
       int64_t(gridDim.x) * blockDim.x);
}

template <int U>
__global__ void __launch_bounds__(kThreads) fused_kernel(const ExtendArgs a) {
  __shared__ int32_t ws[6 * kFusedSeqs + 6];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Scan w = scan_of(ws, a.num_seqs);
  scan_batch(a, w);
  __syncthreads();
  fill<false, U>(a, w, threadIdx.x, kThreads);
}

// ---- release ---------------------------------------------------------------
// One warp per sequence: drops the holds of the finished ones and marks the
// blocks that nothing holds any more in a bitmap of the pool.
__global__ void __launch_bounds__(256) drop_kernel(const ReleaseArgs a) {
  const int s = int((int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (s >= a.num_seqs || !a.finished[s]) return;
  long long L = a.context_lens[s];
  if (L < 0 || L > (long long)a.max_blocks * kBlock) {
    if (lane == 0) flag(a.status, PKV_DEV_BAD_CONTEXT_LEN);
    L = L < 0 ? 0 : (long long)a.max_blocks * kBlock;
  }
  const int nb = int((L + kBlock - 1) / kBlock);
  int32_t* row = a.block_tables + size_t(s) * a.max_blocks;
  for (int j = lane; j < nb; j += 32) {
    const int b = row[j];
    row[j] = -1;
    if (b < 0) continue;  // released before (sliding window)
    if (b >= a.num_blocks) {
      flag(a.status, PKV_DEV_BAD_BLOCK_ID);
      continue;
    }
    bool free_now = true;
    if (a.refcounts) {
      const int old = atomicSub(a.refcounts + b, 1);
      if (old <= 0) {  // nothing held it
        atomicAdd(a.refcounts + b, 1);
        flag(a.status, PKV_DEV_BAD_BLOCK_ID);
      }
      free_now = old == 1;
    }
    if (free_now && (atomicOr(a.bitmap + b / 32, 1u << (b % 32)) >> (b % 32) & 1u))
      flag(a.status, PKV_DEV_BAD_BLOCK_ID);  // two sequences own it without reference counts
  }
  __syncwarp();
  if (lane == 0) a.context_lens[s] = 0;
}

// Pushes the marked blocks onto the free stack in ascending order (whatever
// order the atomics above took). One CTA.
__global__ void __launch_bounds__(kThreads) push_kernel(const ReleaseArgs a) {
  __shared__ int wsum[32][1];
  const int words = (a.num_blocks + 31) / 32;
  int count = *a.free_count;
  __syncthreads();
  if (count < 0 || count > a.num_blocks) {
    if (threadIdx.x == 0) flag(a.status, PKV_DEV_BAD_BLOCK_ID);
    return;
  }
  for (int base = 0; base < words; base += kThreads) {
    const int i = base + threadIdx.x;
    unsigned int m = i < words ? a.bitmap[i] : 0u;
    int v[1] = {__popc(m)}, total[1];
    cta_exclusive<int, 1>(v, wsum, total);
    int at = count + v[0];
    for (; m; m &= m - 1u, ++at) {
      if (at < a.num_blocks) a.free_stack[at] = 32 * i + __ffs(int(m)) - 1;
      else flag(a.status, PKV_DEV_BAD_BLOCK_ID);  // more blocks than the pool has
    }
    count += total[0];
  }
  if (threadIdx.x == 0) *a.free_count = count < a.num_blocks ? count : a.num_blocks;
}

template <typename K, typename A>
cudaError_t launch_after(K kern, unsigned ctas, unsigned threads, cudaStream_t stream, const A& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

size_t extend_workspace_bytes(int num_seqs, int num_slots) {
  if (num_seqs <= kFusedSeqs && num_slots <= kFusedSlots) return 0;
  return (scan_ints(num_seqs) * sizeof(int32_t) + 15) / 16 * 16;
}

cudaError_t launch_extend_block_tables(const ExtendArgs& a, cudaStream_t stream) {
  if (a.num_seqs <= kFusedSeqs && a.num_slots <= kFusedSlots)
    return launch_after(a.num_slots <= kThreads ? fused_kernel<1> : fused_kernel<4>, 1u, unsigned(kThreads), stream, a);
  cudaError_t err = launch_after(scan_kernel, 1u, unsigned(kThreads), stream, a);
  if (err != cudaSuccess) return err;
  const bool many = a.num_slots >= kManySlots;
  const int64_t per = many ? 4 : 2;
  int64_t threads = (int64_t(a.num_slots) + per - 1) / per;
  if (threads < a.num_seqs) threads = a.num_seqs;
  int64_t ctas = (threads + kFillThreads - 1) / kFillThreads;
  if (ctas > 16 * 152) ctas = 16 * 152;  // 16 per SM of a GB300
  return many ? launch_after(fill_kernel<4>, unsigned(ctas), unsigned(kFillThreads), stream, a)
              : launch_after(fill_kernel<2>, unsigned(ctas < 1 ? 1 : ctas), unsigned(kFillThreads), stream, a);
}

cudaError_t launch_release_sequences(const ReleaseArgs& a, cudaStream_t stream) {
  cudaError_t err = cudaMemsetAsync(a.bitmap, 0, release_workspace_bytes(a.num_blocks), stream);
  if (err != cudaSuccess) return err;
  drop_kernel<<<unsigned((int64_t(a.num_seqs) * 32 + 255) / 256), 256, 0, stream>>>(a);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  push_kernel<<<1, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
