// Launch of the decode over the 4-bit KV cache (decode_int4.cuh).
#include "decode_int4.cuh"
#include "decode_launch.cuh"

namespace pkv {
namespace {

constexpr int kInt4Stages = 2;
// Batches of at most kItemCtas items (sequences x KV heads, one wave of CTAs) whose
// tables hold at most kItemPairs pairs of tiles give each item a CTA; the others
// share the list, which starts later and needs a merge but balances. The lengths are
// on the device, so the tables' width decides. Measured for tables of 2048 tokens, item
// against list, in us (groups of 4 query heads, head_dim 128, bf16):
//   about 300 tokens, 8 to 304 items: 5.2 to 8.1, 7.2 to 11.1
//   1000 tokens each: 8 items 8.6, 8.4; 128 10.6, 11.6; 240 11.8, 15.1; 280 12.4, 16.9
//   1000 x e^(0.3 N(0, 1)) tokens, 8 KV heads: 64 items 10.6, 11.2; 96 14.6, 12.0; 128
//   14.2, 12.8; 160 14.7, 13.1; 192 13.6, 13.0; 240 16.7, 14.8; 304 17.0, 18.0; 40 KV
//   heads: 160 10.4, 11.5; 280 14.7, 17.3
// So the rule gives away 5 to 20 % where few sequences of long and mixed lengths make 96
// to 240 items (one CTA ends last), and takes up to 35 % elsewhere; a better one needs
// the lengths. For tables of 8192 tokens (128 items of 5000) 49, 25.
constexpr int64_t kItemCtas = 304;
constexpr int kItemPairs = 64;
// Pairs a warp should have at least, where there are few: one item of 5000 tokens
// 7.4 us (2: 8.4, 4: 10.0), of 30000 10.0 (9.4, 10.1).
constexpr int kMinPairs = 1;

int max_ctas(int head_dim) { return 152 * (head_dim == 256 ? i4_ctas_per_sm<256>() : i4_ctas_per_sm<128>()); }
int warps(int head_dim) { return head_dim == 256 ? i4_warps<256>() : i4_warps<128>(); }

bool item_ctas(int num_seqs, int num_kv_heads, int blocks) {
  return int64_t(num_seqs) * num_kv_heads <= kItemCtas && (blocks + 1) / 2 <= kItemPairs;
}

// CTAs of the list schedule: one wave, fewer where the tables cannot hold
// kMinPairs pairs for every warp.
int list_ctas(int num_seqs, int num_kv_heads, int head_dim, int blocks) {
  const int64_t pairs = int64_t(num_seqs) * num_kv_heads * ((blocks + 1) / 2);
  const int64_t share = warps(head_dim) * kMinPairs, want = (pairs + share - 1) / share;
  return want < max_ctas(head_dim) ? int(want) : max_ctas(head_dim);
}

template <typename T, int D, int H>
cudaError_t launch_int4_dh(const Int4Args& a, cudaStream_t stream) {
  constexpr int NW = i4_warps<D>();
  using C = I4Cfg<D, H, NW, kInt4Stages>;
  static_assert(C::SMEM_BYTES <= 228 * 1024 / i4_ctas_per_sm<D>() - 1024, "CTAs per SM");
  static_assert(sizeof(I4Shared<NW>) <= C::SMEM_BYTES - C::RING_BYTES - C::PIECE_BYTES - C::BAR_BYTES, "shared state");
  auto kern = paged_decode_int4_kernel<T, D, H, NW, kInt4Stages>;
  static bool configured[kMaxDevices] = {};
  cudaError_t err = configure_once(kern, C::SMEM_BYTES, configured);
  if (err != cudaSuccess) return err;
  err = launch_pdl(kern, dim3(unsigned(a.ctas)), dim3(NW * 32), C::SMEM_BYTES, stream, a);
  if (err != cudaSuccess || a.item_ctas || a.ctas == 1) return err;
  return launch_pdl(int4_merge_kernel<T, D>, dim3(unsigned(a.ctas), unsigned(a.group)), dim3(256), 0, stream, a);
}

template <typename T, int D>
cudaError_t launch_int4_d(const Int4Args& a, cudaStream_t stream) {
  return a.group <= 4 ? launch_int4_dh<T, D, 4>(a, stream) : launch_int4_dh<T, D, 8>(a, stream);
}

template <typename T>
cudaError_t launch_int4_t(const Int4Args& a, int head_dim, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_int4_d<T, 64>(a, stream);
    case 128: return launch_int4_d<T, 128>(a, stream);
    case 256: return launch_int4_d<T, 256>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

// Descriptors {item, last CTA} per CTA, then two partial results per CTA: (max,
// sum) and fp32 rows of every query head of a group.
size_t int4_workspace_bytes(int num_seqs, int num_kv_heads, int group, int head_dim, int blocks) {
  if (item_ctas(num_seqs, num_kv_heads, blocks)) return 0;
  const size_t ctas = size_t(list_ctas(num_seqs, num_kv_heads, head_dim, blocks));
  return (ctas * sizeof(int2) + 15) / 16 * 16 + (2 * ctas * group * sizeof(float2) + 15) / 16 * 16 +
         2 * ctas * group * head_dim * sizeof(float);
}

cudaError_t launch_decode_int4(Int4Args a, bool bf16, int head_dim, int blocks, void* workspace, cudaStream_t stream) {
  a.item_ctas = item_ctas(a.num_seqs, a.num_kv_heads, blocks) ? 1 : 0;
  a.ctas = a.item_ctas ? a.num_seqs * a.num_kv_heads : list_ctas(a.num_seqs, a.num_kv_heads, head_dim, blocks);
  if (!a.item_ctas) {
    char* w = static_cast<char*>(workspace);
    a.desc = reinterpret_cast<int2*>(w);
    w += (size_t(a.ctas) * sizeof(int2) + 15) / 16 * 16;
    a.part_ml = reinterpret_cast<float2*>(w);
    w += (size_t(2) * a.ctas * a.group * sizeof(float2) + 15) / 16 * 16;
    a.part_o = reinterpret_cast<float*>(w);
  }
  return bf16 ? launch_int4_t<__nv_bfloat16>(a, head_dim, stream) : launch_int4_t<__half>(a, head_dim, stream);
}

}  // namespace pkv
