// pa_rope.cu -- pa_rope_and_cache and pa_rope_and_cache_fp8: rotate the new
// tokens' queries and keys, write the queries out and the keys and values to
// their slots, in one pass over the rows.  (The rotation: pa_rope.cuh; the FP4
// form: pa_cache_fp4.cu, beside the cache's quantising write.)
//
// HBM bounds a prompt's append, latency a step's: a thread waits for its token's
// slot, position and row of the table and has its items' rows in flight
// meanwhile.  16,381 tokens x (32 + 2 x 8) heads x 128, fp16: 59.6 us for 386 MB,
// 0.95 of the copy rate; 256 tokens x (64 + 2 x 8) x 128 into FP8 caches 3.2 us.
// Three items a thread in flight and four CTAs an SM: with four items and 80
// registers (three CTAs) the prompt takes 65.0 us, with two items 63.7, with four
// items and as many registers as they want (90, two CTAs) 80.5.
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_rope.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;

template <typename T, int D, bool F8>
__global__ void __launch_bounds__(kThreads, 4) rope_and_cache_kernel(const RopeArgs a) {
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
