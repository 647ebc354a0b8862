// Launch of the decode over the 4-bit KV cache (decode_int4.cuh).
#include "decode_int4.cuh"
#include "decode_launch.cuh"

namespace pkv {
namespace {

// Warps per CTA and stages (of two tiles) per warp. Measured on GB300, 128
// dims: 40-head layer, 64 sequences 74.4 us with 4 warps, 78.2 with 2; 32/8
// heads, 256 sequences 26.2 with 4, 22.8 with 2.
template <int H>
constexpr int i4_warps() { return H == 8 ? 2 : 4; }
constexpr int kInt4Stages = 2;

template <typename T, int D, int H>
cudaError_t launch_int4_dh(const DecodeArgs& a, cudaStream_t stream) {
  using C = I4Cfg<D, i4_warps<H>(), kInt4Stages>;
  auto kern = paged_decode_int4_kernel<T, D, H, i4_warps<H>(), kInt4Stages>;
  static bool configured[kMaxDevices] = {};
  cudaError_t err = configure_once(kern, C::SMEM_BYTES, configured);
  if (err != cudaSuccess) return err;
  const dim3 grid(unsigned(a.num_kv_heads), unsigned(a.num_seqs), unsigned(a.max_parts));
  err = launch_pdl(kern, grid, dim3(i4_warps<H>() * 32), C::SMEM_BYTES, stream, a);
  if (err != cudaSuccess) return err;
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_int4_d(const DecodeArgs& a, int gpad, cudaStream_t stream) {
  return gpad <= 2 ? launch_int4_dh<T, D, 2>(a, stream) : launch_int4_dh<T, D, 8>(a, stream);
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
