// pa_attn_fp4.cu -- attention over the FP4 cache, the plainest form: one warp
// for one (query row, query head), one key at a time.
//
//   out = sum_{j <= pos} softmax_j(scale q . K_j) V_j
// with K_j, V_j = g s e2m1(code) read through the block table.  Each lane owns
// head_dim / 32 consecutive dimensions; the dot product is a warp sum, the
// softmax online in fp32 with base 2.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

template <typename T, int D>
__global__ void __launch_bounds__(128) attn_fp4_kernel(const Fp4AttnArgs a) {
  constexpr int kPer = D / 32;  // 2 or 4 dimensions a lane
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int seq = blockIdx.y;
  const int t = static_cast<int>(item / a.num_q_heads), h = static_cast<int>(item % a.num_q_heads);
  int q0 = seq, q_len = 1;
  if (a.query_start) {
    q0 = a.query_start[seq];
    q_len = a.query_start[seq + 1] - q0;
  }
  int ctx = a.context_lens[seq];
  const bool bad = ctx < 0 || ctx > (a.max_blocks_per_seq << a.bs_log2) ||
                   ctx > a.max_context_len ||
                   (a.query_start && (q_len < 0 || q_len > ctx || q_len > a.max_q_len));
  if (bad) {
    if (item == 0 && lane == 0) atomicOr(a.err, kErrBadLen);
    if (a.query_start) return;
    ctx = 0;
  }
  if (t >= q_len) return;
  const int n_keys = ctx - q_len + t + 1;
  const int kvh = h / a.group, bs = 1 << a.bs_log2;
  const int64_t row = (static_cast<int64_t>(q0 + t) * a.num_q_heads + h) * D + lane * kPer;
  float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; e += 2) {
    const float2 v = Elem<T>::unpack(
        *reinterpret_cast<const uint32_t *>(static_cast<const T *>(a.query) + row + e));
    q[e] = v.x;
    q[e + 1] = v.y;
    o[e] = o[e + 1] = 0.f;
  }
  const int32_t *bt = a.block_tables + static_cast<int64_t>(seq) * a.max_blocks_per_seq;
  for (int j = 0; j < n_keys; ++j) {
    const int phys = bt[j >> a.bs_log2];
    if (phys < 0 || phys >= a.num_blocks) {
      if (lane == 0) atomicOr(a.err, kErrBadBlock);
      continue;
    }
    const int64_t tile = (static_cast<int64_t>(phys) * a.num_kv_heads + kvh) * fp4_tile_bytes(bs, D);
    const int r = j & (bs - 1);
    const int64_t at = tile + r * (D / 2) + lane * kPer / 2;
    const int64_t sc = tile + fp4_code_bytes(bs, D) + r * (D / 16) + lane * kPer / 16;
    auto value = [&](const uint8_t *c, float (&x)[kPer]) {
      const float s = e4m3_to_float(c[sc]);
#pragma unroll
      for (int e = 0; e < kPer; e += 2) {
        uint32_t p[4];
        e2m1x8_to_half(c[at + e / 2], p);
        const float2 v = Elem<__half>::unpack(p[0]);
        x[e] = v.x * s;
        x[e + 1] = v.y * s;
      }
    };
    float x[kPer], dot = 0.f;
    value(static_cast<const uint8_t *>(a.k_cache), x);
#pragma unroll
    for (int e = 0; e < kPer; ++e) dot += q[e] * x[e];
#pragma unroll
    for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    const float z = dot * a.scale_log2, mn = fmaxf(m, z);
    const float al = exp2f(m - mn), p = exp2f(z - mn);
    value(static_cast<const uint8_t *>(a.v_cache), x);
    l = l * al + p;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = o[e] * al + p * x[e];
    m = mn;
  }
  const float inv = l > 0.f ? a.out_scale / l : 0.f;
#pragma unroll
  for (int e = 0; e < kPer; e += 2)
    *reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + row + e) =
        Elem<T>::pack(o[e] * inv, o[e + 1] * inv);
}

}  // namespace

cudaError_t launch_attn_fp4(const Fp4AttnArgs &a, int head_dim, int dtype, cudaStream_t stream) {
  const int64_t items = static_cast<int64_t>(a.max_q_len) * a.num_q_heads;
  const dim3 grid(static_cast<unsigned>((items + 3) / 4), a.num_seqs);
  auto kern = dtype == 0 ? (head_dim == 128 ? attn_fp4_kernel<__half, 128> : attn_fp4_kernel<__half, 64>)
                         : (head_dim == 128 ? attn_fp4_kernel<__nv_bfloat16, 128>
                                            : attn_fp4_kernel<__nv_bfloat16, 64>);
  return launch_dependent(kern, grid, dim3(128), 0, stream, a);
}

}  // namespace pa
