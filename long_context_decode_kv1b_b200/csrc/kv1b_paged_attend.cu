// kv1b_paged_attend.cu -- kv1b_paged_attend: the kernel around kv1b_paged_attend.cuh and the merge of what
// the CTAs' ranges cut.
#include "kv1b_paged_attend.cuh"

namespace kv1b {
namespace paged {

template <bool kFine>
__global__ void __launch_bounds__(kThreads, 1) paged_attend_kernel(const PagedAttendParams p, const int G) {
  extern __shared__ __align__(128) uint8_t smem[];
  attend_cta<kFine, false>(p, G, blockIdx.x, smem);
}

// Segments cut by a range boundary: block (c, head) merges the one that starts in CTA c's range and goes
// on past it -- slot 1 of c, then slot 0 of the CTAs after it.
__global__ void __launch_bounds__(128) paged_merge_kernel(const PagedAttendParams p, const int G) {
  __shared__ float2 s_head[kMaxPieces];
  __shared__ float s_max[4];
  pdl_wait();
  const int c = blockIdx.x, hd = blockIdx.y;
  const int2 cut = p.spread[c];
  if (cut.y == 0) return;
  const float* first = p.part + ((static_cast<int64_t>(c) * 2 + 1) * G + hd) * kRow;
  const float* rest = p.part + ((static_cast<int64_t>(c) * 2) * G + hd) * kRow;
  const int64_t step = 2LL * G * kRow;
  merge_pieces(cut.y, [&](int i) { return i == 0 ? first : rest + i * step; }, s_head, s_max, p.out, p.q_dtype,
               (static_cast<int64_t>(cut.x) + hd) * kD);
}

}  // namespace paged
}  // namespace kv1b

using namespace kv1b;

cudaError_t kv1b_launch_paged_pieces(const PagedAttendParams& p, int32_t G, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0}, configured_fine{0};
  const bool fine = p.q_dtype == KV1B_DTYPE_F16;
  const auto kernel = fine ? paged::paged_attend_kernel<true> : paged::paged_attend_kernel<false>;
  cudaError_t e = configure_smem(reinterpret_cast<const void*>(kernel), paged::kSmem, fine ? &configured_fine : &configured);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(p.ncta), dim3(paged::kThreads), paged::kSmem, stream, p, G);
}

cudaError_t kv1b_launch_paged_attend(const PagedAttendParams& p, int32_t G, cudaStream_t stream) {
  const cudaError_t e = kv1b_launch_paged_pieces(p, G, stream);
  if (e != cudaSuccess || p.ncta < 2) return e;
  return launch_pdl(paged::paged_merge_kernel, dim3(p.ncta - 1, G), dim3(128), 0, stream, p, G);
}
