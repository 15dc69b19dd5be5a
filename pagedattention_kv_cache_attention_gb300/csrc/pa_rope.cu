// pa_rope.cu -- pa_rope_and_cache and pa_rope_and_cache_fp8: rotate the new
// tokens' queries and keys, write the queries out and the keys and values to
// their slots, in one pass over the rows.  (The rotation: pa_rope.cuh; the FP4
// form: pa_cache_fp4.cu, beside the cache's quantising write.)
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_rope.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;

template <typename T, int D, bool F8>
__global__ void __launch_bounds__(kThreads) rope_and_cache_kernel(const RopeArgs a) {
  grid_dependency_wait();    // the rows may come from the kernel before
  grid_launch_dependents();  // the next kernel may start its set-up now
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads >> a.group_log2) +
                    (threadIdx.x >> a.group_log2);
  if (t >= a.num_tokens) return;
  rope_token_heads<T, D, F8>(a, t, threadIdx.x & ((1 << a.group_log2) - 1),
                             a.num_q_heads + 2 * a.num_kv_heads);
}

template <typename T, int D, bool F8>
cudaError_t launch(RopeArgs a, cudaStream_t stream) {
  a.group_log2 = rope_group_log2((a.num_q_heads + 2 * a.num_kv_heads) * (D / 16));
  const int64_t per_cta = kThreads >> a.group_log2;
  return launch_dependent(rope_and_cache_kernel<T, D, F8>,
                          dim3(static_cast<unsigned>((a.num_tokens + per_cta - 1) / per_cta)),
                          dim3(kThreads), 0, stream, a);
}

template <typename T, int D>
cudaError_t launch_t(const RopeArgs &a, bool to_fp8, cudaStream_t stream) {
  return to_fp8 ? launch<T, D, true>(a, stream) : launch<T, D, false>(a, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int head_dim, int dtype, bool to_fp8,
                        cudaStream_t stream) {
  if (dtype == 0)
    return head_dim == 128 ? launch_t<__half, 128>(a, to_fp8, stream)
                           : launch_t<__half, 64>(a, to_fp8, stream);
  return head_dim == 128 ? launch_t<__nv_bfloat16, 128>(a, to_fp8, stream)
                         : launch_t<__nv_bfloat16, 64>(a, to_fp8, stream);
}

}  // namespace pa
