// Host-side launchers of the CUDA kernels (internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace pkv {

struct DecodeArgs;
struct SkArgs;

constexpr int kMaxParts = 8192;   // split-K partitions per sequence (merge smem bound)
constexpr int kMaxDevices = 64;

// Decode. head_dim in {64,128,256}; gpad in {1,2,4,8}. gpad 1 runs the CUDA-core
// kernel; gpad >= 2 runs the tensor-core kernel, which reads the pools through
// the tensor maps kmap/vmap: three each, 128-byte swizzle, boxes of 16, 8 and
// 4 rows x 64 columns (the balanced schedule reads the first of each).
cudaError_t launch_decode_f16(const DecodeArgs& a, int head_dim, int gpad, const CUtensorMap* kmap,
                              const CUtensorMap* vmap, cudaStream_t stream);
cudaError_t launch_decode_bf16(const DecodeArgs& a, int head_dim, int gpad, const CUtensorMap* kmap,
                               const CUtensorMap* vmap, cudaStream_t stream);

// The same grids over the tails of sequences (DecodeArgs::query_rows, from, join_ml, join_o).
cudaError_t launch_decode_tail(const DecodeArgs& a, bool bf16, int head_dim, int gpad, const CUtensorMap* kmap,
                               const CUtensorMap* vmap, cudaStream_t stream);

// Decode with the balanced persistent schedule (decode_sk.cuh); same gpad rules.
cudaError_t launch_decode_sk_f16(const SkArgs& a, int head_dim, int gpad, const CUtensorMap* kmap,
                                 const CUtensorMap* vmap, cudaStream_t stream);
cudaError_t launch_decode_sk_bf16(const SkArgs& a, int head_dim, int gpad, const CUtensorMap* kmap,
                                  const CUtensorMap* vmap, cudaStream_t stream);

// Largest batch the balanced schedule takes for these sizes (its prefix sums
// share the CTA's shared memory with the rings); 0 for unsupported sizes.
int decode_sk_max_seqs(int head_dim, int gpad);

// The launch plan of a batch (num_seqs <= 1024) into `plan`: a 16-byte header
// {magic, num_seqs, 0, 0}, then the long-first order int32[num_seqs] (grid row
// -> sequence; the shortest sequences last with short_last); with `rows`, also
// int4[2 * num_seqs] per rank {sequence, length, ids 0..5 of `tables`} (the
// sequence -1 when tables is null).
cudaError_t launch_seq_order(const int32_t* lens, int num_seqs, int max_len, int window, bool short_last,
                             int4* plan, const int32_t* tables, int max_blocks, int4* rows, cudaStream_t stream);

// The prefix plan of the shared-prefix schedule (decode_prefix.cuh): header,
// groups int4[num_seqs / 2], chunks int4[num_seqs], the sequences outside any
// group int32[num_seqs], and the merge counters [num_seqs][num_kv_heads]
// zeroed. num_seqs <= 1024, tables of at most 256 blocks; groups of at most
// max_members sequences; slots = CTAs the decode grid holds at once.
cudaError_t launch_prefix_plan(const int32_t* lens, const int32_t* tables, int num_seqs, int max_blocks,
                               int num_kv_heads, int slots, int max_members, int4* header, int4* groups, int4* chunks,
                               int32_t* others, unsigned int* counters, cudaStream_t stream);
// CTAs of the shared-prefix decode grid (head_dim 64/128/256) resident at once on the current device.
cudaError_t prefix_resident_ctas(int head_dim, int* ctas);
// One warp that waits on an mbarrier no copy completes (bounded-wait self-test).
cudaError_t launch_bounded_wait_selftest(unsigned long long limit_ns, unsigned int* status, cudaStream_t stream);
cudaError_t launch_trace_stamp(unsigned long long* dst, cudaStream_t stream);

// Bit copies; element size is 2 bytes for both supported dtypes.
cudaError_t launch_reshape_and_cache(const void* k, const void* v, void* k_pool, void* v_pool,
                                     const int64_t* slots, int num_tokens, int num_kv_heads,
                                     int head_dim, int num_blocks, unsigned int* status,
                                     cudaStream_t stream);
cudaError_t launch_copy_blocks(void* k_pool, void* v_pool, const int64_t* pairs, int num_pairs,
                               int num_kv_heads, int head_dim, int num_blocks,
                               unsigned int* status, cudaStream_t stream);
// Block copy of two pools whose blocks are bytes_per_block bytes (a multiple of 16).
cudaError_t launch_copy_blocks_bytes(void* k_pool, void* v_pool, const int64_t* pairs, int num_pairs,
                                     int64_t bytes_per_block, int num_blocks, unsigned int* status,
                                     cudaStream_t stream);

// INT8 KV cache: quantising cache write (head_dim 64, 128 or 256) and decode
// over int8 codes with per-row fp32 scales. The tensor-core kernel reads the
// code pools through uint8 tensor maps (boxes of 16 rows x min(D, 128) bytes,
// 128-byte swizzle, 64-byte at D = 64); decode_int8_uses_tensor_maps() says
// whether the build needs them.
cudaError_t launch_reshape_and_cache_int8(const void* k, const void* v, bool bf16, int8_t* k_codes,
                                          int8_t* v_codes, float* k_scale, float* v_scale, const int64_t* slots,
                                          int num_tokens, int num_kv_heads, int head_dim, int num_blocks,
                                          unsigned int* status, cudaStream_t stream);
bool decode_int8_uses_tensor_maps();
cudaError_t launch_decode_int8(const DecodeArgs& a, bool bf16, int head_dim, int gpad, const CUtensorMap* kmap,
                               const CUtensorMap* vmap, cudaStream_t stream);

// 4-bit KV cache (int4_layout.cuh): quantising write, or read back of the rows
// at `slots` into k and v (gather); decode.
cudaError_t launch_cache_int4(bool gather, void* k, void* v, bool bf16, void* cache, const int64_t* slots,
                              int num_tokens, int num_kv_heads, int head_dim, int num_blocks, unsigned int* status,
                              cudaStream_t stream);
struct Int4Args {
  void* out;
  const void* q;
  const void* cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  unsigned int* status;
  int num_seqs, num_q_heads, num_kv_heads;
  int group;           // query heads per KV head
  int max_blocks_per_seq, num_blocks;
  int window;          // attend over the last `window` tokens (0 = all)
  float scale_log2;    // scale * log2(e)
  // set by the launcher: CTAs, whether each takes one item, and the workspace's parts
  int ctas, item_ctas;
  int2* desc;
  float2* part_ml;
  float* part_o;
};
// `blocks`: the most table entries of a sequence that a call reads (fewer with a window).
size_t int4_workspace_bytes(int num_seqs, int num_kv_heads, int group, int head_dim, int blocks);
cudaError_t launch_decode_int4(Int4Args a, bool bf16, int head_dim, int blocks, void* workspace, cudaStream_t stream);
// Block copy of one pool whose blocks are bytes_per_block bytes (a multiple of 16).
cudaError_t launch_copy_blocks_pool(void* pool, const int64_t* pairs, int num_pairs, int64_t bytes_per_block,
                                    int num_blocks, unsigned int* status, cudaStream_t stream);

// Latent attention: rows of kLatentDim latent and kRopeDim rotary elements.
constexpr int kLatentDim = 512;
constexpr int kRopeDim = 64;
constexpr int kLatentRow = kLatentDim + kRopeDim;

struct LatentArgs {
  void* out;
  const void* q;
  const void* cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  unsigned int* status;
  void* workspace;
  int num_seqs;
  int num_heads;
  int max_blocks_per_seq;
  int num_blocks;
  float scale_log2;  // scale * log2(e)
  // set by the launcher: work ranges, blocks of heads, heads per block, and the workspace's parts
  int ranges, head_blocks, block_heads, desc_by_seq;
  int2* desc;
  float2* part_ml;
  float* part_o;
};

cudaError_t launch_latent_write(const void* latent, const void* rope, void* cache, const int64_t* slots,
                                int num_tokens, int64_t latent_stride, int64_t rope_stride, int num_blocks,
                                unsigned int* status, cudaStream_t stream);
size_t latent_workspace_bytes(int num_seqs, int num_heads, int max_blocks_per_seq);
// Rows of the query's tensor-map box (query heads a CTA takes, padded).
int latent_query_box(int num_seqs, int num_heads, int max_blocks_per_seq);
// cache_map: the cache as {64 elements, 8 rows, 9 chunks, 2 * num_blocks
// groups}, boxes of one block; q_map: q as [num_seqs, num_heads, 576], boxes of
// 1 x latent_query_box x 64; both with the 128-byte swizzle and zero fill.
cudaError_t launch_latent_decode(const LatentArgs& a, bool bf16, const CUtensorMap& cache_map,
                                 const CUtensorMap& q_map, cudaStream_t stream);

// The cache write that rotates queries and keys (rotary.cu).
struct RotaryArgs {
  void* q_out;
  const void* q;
  const void* k;
  const void* v;
  int64_t q_out_stride, q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t* positions;
  const float* cos_sin;  // [max_positions][rotary_dim]
  void* k_pool;
  void* v_pool;
  const int64_t* slots;
  unsigned int* status;
  int num_tokens, num_q_heads, num_kv_heads, head_dim, num_blocks;
  int max_positions, rotary_dim, interleaved;
};
cudaError_t launch_rotary(const RotaryArgs& a, bool bf16, cudaStream_t stream);

// Attention of several query tokens per sequence, and of sequences that share a
// prefix, over the paged cache (prompt.cuh).
struct PromptArgs {
  void* out;
  const void* q;
  const void* k_pool;
  const void* v_pool;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_starts;   // [num_seqs + 1]; null: one query per sequence
  const int32_t* group_starts;   // [num_groups + 1], and
  const int32_t* prefix_blocks;  // [num_groups]: sequences that share their first blocks (num_groups 0: none)
  unsigned int* status;
  int num_seqs, num_tokens, num_groups;
  int num_q_heads, num_kv_heads;
  int group;         // query heads per KV head
  int max_blocks_per_seq, num_blocks;
  int causal;
  int window;        // causal: attend over the last `window` tokens (0 = all)
  float scale_log2;  // scale * log2(e)
  int tails;         // a decode grid takes sequences with one query token (prompts), and what follows the prefixes, but
                     // for the longest
  // set by the launcher: query tokens of a tile of rows and of a block, CTAs, rows of a
  // slot of partial results, and the workspace's parts
  int tile_tokens, block_tokens, shares;
  size_t slot_rows;
  int4* desc;   // per share, the item that starts in it and goes on past it (prompts)
  int2* link;   // per item, the shares that hold its pieces (prefix decode)
  int* more;    // per share, whether it begins inside an item
  float2* part_ml;
  float* part_o;
  int32_t* from;  // per sequence, where its prefix ends (prefix decode with tails)
  int* limit;     // positions up to which the decode grid takes a single token (tails)
};
// What a tail grid reads of the workspace: the limit; behind prefixes from, and their partial
// results per (sequence, query head).
struct PromptTails {
  const int* limit;
  const int32_t* from;
  const float2* ml;
  const float* o;
};
PromptTails prompt_tails(PromptArgs a, int head_dim, void* workspace);
// Query tokens of one copy of Q (128 rows): the second box size of its tensor map.
inline int prompt_tile_tokens(int group) { return 128 / group; }
size_t prompt_workspace_bytes(const PromptArgs& a, int head_dim);
// Tensor maps of a call, with the 128-byte swizzle and zero fill: q as {64 elements,
// heads, tokens, head_dim / 64 chunks}, in boxes of one KV head's query heads x
// prompt_tile_tokens (q) or 1 token (q1); the pools as {64 elements, 8 rows, head_dim /
// 64 chunks, 8-row groups}, in boxes of one (block, KV head).
struct PromptMaps {
  CUtensorMap q, q1, k, v;
};
cudaError_t launch_prompt(PromptArgs a, bool bf16, int head_dim, void* workspace, const PromptMaps& maps,
                          cudaStream_t stream);

// Block tables on the device (tables.cu).
struct ExtendArgs {
  int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* new_tokens;
  const int32_t* free_stack;
  const int32_t* free_count;
  int32_t* refcounts;       // or null: nothing is shared
  int32_t* new_lens;        // may be context_lens
  int32_t* new_free_count;  // may be free_count
  int64_t* slot_mapping;
  int64_t* cow_pairs;       // [S][2], with refcounts
  int32_t* info;            // {flags, tokens, blocks, pairs}, or null
  int32_t* workspace;       // extend_workspace_bytes
  unsigned int* status;
  int num_seqs;
  int max_blocks;
  int num_blocks;
  int num_slots;
  int slots_aligned;        // slot_mapping is 16-byte aligned
};

struct ReleaseArgs {
  int32_t* block_tables;
  int32_t* context_lens;
  const int32_t* finished;
  int32_t* free_stack;
  int32_t* free_count;
  int32_t* refcounts;  // or null
  unsigned int* bitmap;
  unsigned int* status;
  int num_seqs;
  int max_blocks;
  int num_blocks;
};

size_t extend_workspace_bytes(int num_seqs, int num_slots);
inline size_t release_workspace_bytes(int num_blocks) { return (size_t(num_blocks) + 31) / 32 * 4; }
cudaError_t launch_extend_block_tables(const ExtendArgs& a, cudaStream_t stream);
cudaError_t launch_release_sequences(const ReleaseArgs& a, cudaStream_t stream);

}  // namespace pkv
