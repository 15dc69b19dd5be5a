// pa_cache_fp4.cu -- the FP4 cache's quantising write and its read-back.
//
// Write, for 16 elements x of a token's K or V row (g: the cache's scale):
//   s    = e4m3(max|x| / (6 g))     6 is the largest E2M1 magnitude
//   z    = s g,   code = e2m1(x (1 / z))
// with an IEEE fp32 quotient for the scale and one IEEE fp32 reciprocal for
// the 16 codes (a division for every element would be eight instructions or
// so for each; the reciprocal moves a quotient by at most an ulp or two of
// fp32, which matters only next to a tie).  s = 0 stores zeros (the whole
// group is below half of g * 2^-9 * 6); a NaN in the group stores the NaN
// scale and zero codes, so that the group reads back as NaN.
// Read: code * (s g) in fp32, rounded once to the output type.
//
// One thread takes one group of 16: 32 bytes of the 16-bit row, 8 bytes of
// codes and one scale byte.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kThreads = 128;

// Place of (token at `slot`, head h, group b) in a cache: its codes' and its
// scale's byte offset.
__device__ __forceinline__ void fp4_place(const Fp4CacheArgs &a, int64_t slot, int h, int b,
                                          int64_t &codes, int64_t &scale) {
  const int64_t blk = slot >> a.bs_log2;
  const int row = static_cast<int>(slot) & ((1 << a.bs_log2) - 1);
  const int bs = 1 << a.bs_log2;
  const int64_t tile = (blk * a.num_kv_heads + h) * fp4_tile_bytes(bs, a.head_dim);
  codes = tile + row * (a.head_dim / 2) + b * 8;
  scale = tile + fp4_code_bytes(bs, a.head_dim) + row * (a.head_dim / 16) + b;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) cache_fp4_write_kernel(const Fp4CacheArgs a) {
  grid_dependency_wait();    // rows and slots may come from the kernel before
  grid_launch_dependents();  // the next kernel may start its set-up now
  const int groups = a.head_dim / kFp4Group;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t per_token = static_cast<int64_t>(a.num_kv_heads) * groups;
  if (i >= a.num_tokens * per_token) return;
  const int64_t t = i / per_token;
  const int u = static_cast<int>(i - t * per_token), h = u / groups, b = u % groups;
  const int64_t slot = a.slot_mapping[t];
  if (slot < 0) return;
  if (slot >= (a.num_blocks << a.bs_log2)) {
    if (u == 0) atomicOr(a.err, kErrBadSlot);
    return;
  }
  const bool is_v = blockIdx.y != 0;
  const T *row = static_cast<const T *>(is_v ? a.value : a.key) +
                 t * (is_v ? a.value_stride : a.key_stride) + static_cast<int64_t>(u) * kFp4Group;
  const float g = is_v ? a.v_scale : a.k_scale;
  const uint4 x0 = reinterpret_cast<const uint4 *>(row)[0];
  const uint4 x1 = reinterpret_cast<const uint4 *>(row)[1];
  float x[16];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float2 lo = Elem<T>::unpack(word_of(x0, w)), hi = Elem<T>::unpack(word_of(x1, w));
    x[2 * w] = lo.x;
    x[2 * w + 1] = lo.y;
    x[8 + 2 * w] = hi.x;
    x[8 + 2 * w + 1] = hi.y;
  }
  float top = 0.f;
  bool nan = false;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    top = fmaxf(top, fabsf(x[e]));
    nan |= x[e] != x[e];
  }
  uint32_t s = nan ? kFp4NanScale : float_to_e4m3(__fdiv_rn(top, __fmul_rn(6.f, g)));
  const float z = __fmul_rn(e4m3_to_float(s), g);
  const float inv = __frcp_rn(z);
  uint32_t lo = 0, hi = 0;
  if (!nan && s != 0) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __fmul_rn(x[e], inv);
    lo = float8_to_e2m1x8(y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __fmul_rn(x[8 + e], inv);
    hi = float8_to_e2m1x8(y);
  }
  int64_t codes, scale;
  fp4_place(a, slot, h, b, codes, scale);
  uint8_t *cache = static_cast<uint8_t *>(is_v ? a.v_cache : a.k_cache);
  *reinterpret_cast<uint2 *>(cache + codes) = make_uint2(lo, hi);
  cache[scale] = static_cast<uint8_t>(s);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) cache_fp4_read_kernel(const Fp4CacheArgs a) {
  grid_dependency_wait();  // the pool and the slots may come from the kernel before
  grid_launch_dependents();
  const int groups = a.head_dim / kFp4Group;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t per_token = static_cast<int64_t>(a.num_kv_heads) * groups;
  if (i >= a.num_tokens * per_token) return;
  const int64_t t = i / per_token;
  const int u = static_cast<int>(i - t * per_token), h = u / groups, b = u % groups;
  const int64_t slot = a.slot_mapping[t];
  if (slot < 0) return;
  if (slot >= (a.num_blocks << a.bs_log2)) {
    if (u == 0) atomicOr(a.err, kErrBadSlot);
    return;
  }
  const bool is_v = blockIdx.y != 0;
  int64_t codes, scale;
  fp4_place(a, slot, h, b, codes, scale);
  const uint8_t *cache = static_cast<const uint8_t *>(is_v ? a.v_cache : a.k_cache);
  const uint2 w = *reinterpret_cast<const uint2 *>(cache + codes);
  const float z = __fmul_rn(e4m3_to_float(cache[scale]), is_v ? a.v_scale : a.k_scale);
  uint32_t e0[4], e1[4], o[8];
  e2m1x8_to_half(w.x, e0);
  e2m1x8_to_half(w.y, e1);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 p = Elem<__half>::unpack(e0[k]), q = Elem<__half>::unpack(e1[k]);
    o[k] = Elem<T>::pack(__fmul_rn(p.x, z), __fmul_rn(p.y, z));
    o[4 + k] = Elem<T>::pack(__fmul_rn(q.x, z), __fmul_rn(q.y, z));
  }
  T *row = static_cast<T *>(is_v ? a.value : a.key) +
           t * (is_v ? a.value_stride : a.key_stride) + static_cast<int64_t>(u) * kFp4Group;
  reinterpret_cast<uint4 *>(row)[0] = make_uint4(o[0], o[1], o[2], o[3]);
  reinterpret_cast<uint4 *>(row)[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

dim3 cache_grid(const Fp4CacheArgs &a) {
  const int64_t n = static_cast<int64_t>(a.num_tokens) * a.num_kv_heads * (a.head_dim / kFp4Group);
  return dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads), 2);
}

}  // namespace

cudaError_t launch_cache_fp4_write(const Fp4CacheArgs &a, int dtype, cudaStream_t stream) {
  return launch_dependent(dtype == 0 ? cache_fp4_write_kernel<__half>
                                     : cache_fp4_write_kernel<__nv_bfloat16>,
                          cache_grid(a), dim3(kThreads), 0, stream, a);
}

cudaError_t launch_cache_fp4_read(const Fp4CacheArgs &a, int dtype, cudaStream_t stream) {
  return launch_dependent(dtype == 0 ? cache_fp4_read_kernel<__half>
                                     : cache_fp4_read_kernel<__nv_bfloat16>,
                          cache_grid(a), dim3(kThreads), 0, stream, a);
}

}  // namespace pa
