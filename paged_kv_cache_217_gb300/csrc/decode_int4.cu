// Launch of the decode over the 4-bit KV cache (decode_int4.cuh).
#include "decode_int4.cuh"
#include "decode_launch.cuh"

namespace pkv {
namespace {

constexpr int kInt4Warps = 4;
constexpr int kInt4Stages = 4;

template <typename T, int D, int G>
cudaError_t launch_int4_dg(const DecodeArgs& a, cudaStream_t stream) {
  using C = I4Cfg<D, kInt4Warps, kInt4Stages>;
  auto kern = paged_decode_int4_kernel<T, D, G, kInt4Warps, kInt4Stages>;
  static bool configured[kMaxDevices] = {};
  cudaError_t err = configure_once(kern, C::SMEM_BYTES, configured);
  if (err != cudaSuccess) return err;
  const dim3 grid(unsigned(a.num_kv_heads), unsigned(a.num_seqs), unsigned(a.max_parts));
  err = launch_pdl(kern, grid, dim3(kInt4Warps * 32), C::SMEM_BYTES, stream, a);
  if (err != cudaSuccess) return err;
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_int4_d(const DecodeArgs& a, int gpad, cudaStream_t stream) {
  return gpad == 1 ? launch_int4_dg<T, D, 1>(a, stream) : launch_int4_dg<T, D, 8>(a, stream);
}

template <typename T>
cudaError_t launch_int4_t(const DecodeArgs& a, int head_dim, int gpad, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_int4_d<T, 64>(a, gpad, stream);
    case 128: return launch_int4_d<T, 128>(a, gpad, stream);
    case 256: return launch_int4_d<T, 256>(a, gpad, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_decode_int4(const DecodeArgs& a, bool bf16, int head_dim, int gpad, cudaStream_t stream) {
  return bf16 ? launch_int4_t<__nv_bfloat16>(a, head_dim, gpad, stream)
              : launch_int4_t<__half>(a, head_dim, gpad, stream);
}

}  // namespace pkv
