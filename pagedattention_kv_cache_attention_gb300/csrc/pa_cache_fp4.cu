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
// A warp takes a token (or several tokens of few heads), K and V, and a lane 8
// elements at a time: 16 bytes of the 16-bit row and 4 bytes of codes, so that
// a warp's loads and stores are whole lines on both sides.  Two neighbours
// share a group.  The token's slot, tile and row are worked out once for the
// warp: with a thread for a group and 64-bit arithmetic of its own the kernels
// were bound by instructions (a prompt of 16,381 tokens x 8 heads x 128 written
// and read back in 39 us, 65,536 tokens read in 69 us; these take 33.5 and 55).
// Apart, the prompt's write takes 20 us and its read-back 16, of 12.7 us each for
// their bytes: loads in flight bound them (the write has 80 registers and issues in
// 44 % of the cycles), and on the long read HBM, at 0.92 of the copy rate.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"
#include "pa_rope.cuh"

#ifndef PA_CACHE_FP4_BATCH
#define PA_CACHE_FP4_BATCH 4
#endif
#ifndef PA_CACHE_FP4_CTAS
#define PA_CACHE_FP4_CTAS 1000
#endif

namespace pa {

namespace {

constexpr int kWarps = 8;
constexpr int kBatch = PA_CACHE_FP4_BATCH;  // items of K and of V that a lane has in flight

// Calls body(token, slot, item0) for the tokens of this warp: a lane's items
// are item0, item0 + 32, ... below Hkv * D / 8 (none if item0 is not).
// (ctas: the CTAs that share the tokens)
template <int D, typename Args, typename F>
__device__ __forceinline__ void for_tokens(const Args &a, unsigned ctas, F &&body) {
  const int lane = threadIdx.x & 31, items = a.num_kv_heads * (D / 8);
  const int per_warp = items < 32 ? 32 / items : 1;  // tokens that a warp takes at once
  const int sub = items < 32 ? lane / items : 0;
  const int item0 = sub < per_warp ? lane - sub * items : items;
  const int64_t step = static_cast<int64_t>(ctas) * kWarps * per_warp;
  for (int64_t t = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * per_warp;
       t < a.num_tokens; t += step) {
    const int64_t token = t + sub;
    int64_t slot = sub < per_warp && token < a.num_tokens ? a.slot_mapping[token] : -1;
    if constexpr (std::is_same<Args, RopeArgs>::value) {
      if (slot >= 0 && !rope_token(a, slot, a.positions[token], item0 == 0)) slot = -1;
    } else if (slot >= (a.num_blocks << a.bs_log2)) {
      if (item0 == 0) atomicOr(a.err, kErrBadSlot);
      slot = -1;
    }
    body(token, slot, slot < 0 ? items : item0);
  }
}

// Where the codes and the scale of a lane's item lie in the cache, from the
// token's first tile on; 32 items further they lie `step` bytes on (32 items
// are two or four heads).
template <int D> struct Place {
  int codes, scale, step;
  int64_t tile0;
  template <typename Args>
  __device__ __forceinline__ Place(const Args &a, int64_t slot, int item0) {
    constexpr int kPerHead = D / 8;
    const int bs = 1 << a.bs_log2, row = static_cast<int>(slot) & (bs - 1);
    const int h = item0 / kPerHead, b = item0 % kPerHead;
    tile0 = (slot >> a.bs_log2) * a.num_kv_heads * fp4_tile_bytes(bs, D);
    codes = h * fp4_tile_bytes(bs, D) + row * (D / 2) + b * 4;
    scale = h * fp4_tile_bytes(bs, D) + fp4_code_bytes(bs, D) + row * (D / 16) + b / 2;
    step = 32 / kPerHead * fp4_tile_bytes(bs, D);
  }
};

// Larger of two pairs of 16-bit magnitudes, NaN if either is.
template <typename T> __device__ __forceinline__ uint32_t max2_nan(uint32_t x, uint32_t y) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 m = __hmax2_nan(*reinterpret_cast<const __half2 *>(&x),
                                  *reinterpret_cast<const __half2 *>(&y));
    return *reinterpret_cast<const uint32_t *>(&m);
  } else {
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&x),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&y));
    return *reinterpret_cast<const uint32_t *>(&m);
  }
}
// Largest magnitude of even and of odd elements of 8.
template <typename T> __device__ __forceinline__ uint32_t top2(const uint4 &x) {
  constexpr uint32_t kMag = 0x7fff7fffu;
  return max2_nan<T>(max2_nan<T>(x.x & kMag, x.y & kMag), max2_nan<T>(x.z & kMag, x.w & kMag));
}
// 8 elements times inv to 8 codes.
template <typename T> __device__ __forceinline__ uint32_t codes8(const uint4 &raw, float inv) {
  float y[8];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float2 v = Elem<T>::unpack(word_of(raw, w));
    y[2 * w] = __fmul_rn(v.x, inv);
    y[2 * w + 1] = __fmul_rn(v.y, inv);
  }
  return float8_to_e2m1x8(y);
}

// 8 elements of a K and of a V row, the lane's halves of a group each, to
// codes and the group's scales.  The even lane of a pair works out K's scale
// and reciprocal, the odd one V's.
template <typename T>
__device__ __forceinline__ void quantise8(const uint4 &k, const uint4 &v, float g, uint32_t &kq,
                                          uint32_t &vq, uint32_t &scale) {
  const uint32_t tk = top2<T>(k), tv = top2<T>(v);
  uint32_t top = max2_nan<T>(__byte_perm(tk, tv, 0x5410), __byte_perm(tk, tv, 0x7632));
  top = max2_nan<T>(top, __shfl_xor_sync(0xffffffffu, top, 1));  // (K, V) of the whole group
  const bool odd = threadIdx.x & 1;
  const float2 both = Elem<T>::unpack(top);
  scale = float_to_e4m3(__fdiv_rn(odd ? both.y : both.x, __fmul_rn(6.f, g)));  // NaN stays NaN
  const float inv = __frcp_rn(__fmul_rn(e4m3_to_float(scale), g));
  const bool none = scale == 0 || scale == kFp4NanScale;  // zero codes
  const float inv_o = __shfl_xor_sync(0xffffffffu, inv, 1);
  const bool none_o = __shfl_xor_sync(0xffffffffu, none ? 1 : 0, 1) != 0;
  kq = (odd ? none_o : none) ? 0u : codes8<T>(k, odd ? inv_o : inv);
  vq = (odd ? none : none_o) ? 0u : codes8<T>(v, odd ? inv : inv_o);
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) cache_fp4_write_kernel(const Fp4CacheArgs a) {
  grid_dependency_wait();    // rows and slots may come from the kernel before
  grid_launch_dependents();  // the next kernel may start its set-up now
  const int items = a.num_kv_heads * (D / 8);
  const bool odd = threadIdx.x & 1;
  for_tokens<D>(a, gridDim.x, [&](int64_t token, int64_t slot, int item0) {
    const uint4 *key = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.key) +
                                                       token * a.key_stride);
    const uint4 *value = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.value) +
                                                         token * a.value_stride);
    const Place<D> at(a, slot, item0);
    uint8_t *kc = static_cast<uint8_t *>(a.k_cache) + at.tile0;
    uint8_t *vc = static_cast<uint8_t *>(a.v_cache) + at.tile0;
    // (every lane of the warp runs through: neighbours shuffle)
    for (int i0 = 0; i0 < items; i0 += 32 * kBatch) {
      uint4 k[kBatch], v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int item = item0 + i0 + 32 * i;
        k[i] = item < items ? key[item] : make_uint4(0, 0, 0, 0);
        v[i] = item < items ? value[item] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (i0 + 32 * i >= items) break;
        const int off = (i0 / 32 + i) * at.step;
        uint32_t kq, vq, scale;
        quantise8<T>(k[i], v[i], odd ? a.v_scale : a.k_scale, kq, vq, scale);
        if (item0 + i0 + 32 * i < items) {
          *reinterpret_cast<uint32_t *>(kc + at.codes + off) = kq;
          *reinterpret_cast<uint32_t *>(vc + at.codes + off) = vq;
          (odd ? vc : kc)[at.scale + off] = static_cast<uint8_t>(scale);
        }
      }
    }
  });
}

// pa_rope_and_cache_fp4.  The first `kv_ctas` CTAs write K and V as above, with
// each lane's chunk of K rotated on the way: it needs the chunk that holds the
// other elements of its pairs (nothing where pairs are neighbours), which another
// lane of the warp loads too, so the second load comes out of L1.  The other CTAs
// rotate the queries.  Loads in flight bound it: 16,381 tokens x (32 + 2 x 8) heads x
// 128, fp16, 65 us for 319 MB (floor 47); 74 with three CTAs an SM in place of four
// (80 registers), 67 with one item a lane in flight in place of two.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, 4) cache_fp4_rope_kernel(const RopeArgs a,
                                                                     const unsigned kv_ctas) {
  constexpr int kTake = 2;   // items of K and of V that a lane has in flight
  grid_dependency_wait();    // rows and slots may come from the kernel before
  grid_launch_dependents();  // the next kernel may start its set-up now
  if (blockIdx.x >= kv_ctas) {
    const int64_t t = static_cast<int64_t>(blockIdx.x - kv_ctas) * (kWarps * 32 >> a.group_log2) +
                      (threadIdx.x >> a.group_log2);
    if (t < a.num_tokens)
      rope_token_heads<T, D, false>(a, t, threadIdx.x & ((1 << a.group_log2) - 1), a.num_q_heads);
    return;
  }
  const int items = a.num_kv_heads * (D / 8);
  const bool odd = threadIdx.x & 1;
  for_tokens<D>(a, kv_ctas, [&](int64_t token, int64_t slot, int item0) {
    const uint4 *key = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.key) +
                                                       token * a.key_stride);
    const uint4 *value = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.value) +
                                                         token * a.value_stride);
    const Place<D> at(a, slot, item0);
    uint8_t *kc = static_cast<uint8_t *>(a.k_cache) + at.tile0;
    uint8_t *vc = static_cast<uint8_t *>(a.v_cache) + at.tile0;
    // chunk b of its head: pairs with chunk b + other, cosines and sines of its
    // 8 elements (negated sines where the element is the pair's first)
    const int b = item0 % (D / 8), half = a.rotary_dim / 16;
    const bool turn = item0 < items && b < 2 * half;
    const int other = a.interleaved || !turn ? 0 : b < half ? half : -half;
    float c[8], s[8];
    if (turn) {
      const float *row = a.cos_sin + a.positions[token] * a.rotary_dim;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int pair = a.interleaved ? 4 * b + i / 2 : 8 * (b < half ? b : b - half) + i;
        c[i] = row[pair];
        s[i] = row[a.rotary_dim / 2 + pair];
      }
    }
    // (every lane of the warp runs through: neighbours shuffle)
    for (int i0 = 0; i0 < items; i0 += 32 * kTake) {
      uint4 k[kTake], p[kTake], v[kTake];
#pragma unroll
      for (int i = 0; i < kTake; ++i) {
        const int item = item0 + i0 + 32 * i;
        k[i] = item < items ? key[item] : make_uint4(0, 0, 0, 0);
        p[i] = item < items ? key[item + other] : make_uint4(0, 0, 0, 0);
        v[i] = item < items ? value[item] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kTake; ++i) {
        if (i0 + 32 * i >= items) break;
        if (turn) {
          uint32_t w4[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 x = Elem<T>::unpack(word_of(k[i], w)), y = Elem<T>::unpack(word_of(p[i], w));
            float lo, hi, unused;
            if (a.interleaved) {
              rope_pair(x.x, x.y, c[2 * w], s[2 * w], lo, hi);
            } else if (b < half) {
              rope_pair(x.x, y.x, c[2 * w], s[2 * w], lo, unused);
              rope_pair(x.y, y.y, c[2 * w + 1], s[2 * w + 1], hi, unused);
            } else {
              rope_pair(y.x, x.x, c[2 * w], s[2 * w], unused, lo);
              rope_pair(y.y, x.y, c[2 * w + 1], s[2 * w + 1], unused, hi);
            }
            w4[w] = Elem<T>::pack(lo, hi);
          }
          k[i] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
        const int off = (i0 / 32 + i) * at.step;
        uint32_t kq, vq, scale;
        quantise8<T>(k[i], v[i], odd ? a.v_scale : a.k_scale, kq, vq, scale);
        if (item0 + i0 + 32 * i < items) {
          *reinterpret_cast<uint32_t *>(kc + at.codes + off) = kq;
          *reinterpret_cast<uint32_t *>(vc + at.codes + off) = vq;
          (odd ? vc : kc)[at.scale + off] = static_cast<uint8_t>(scale);
        }
      }
    }
  });
}

// 8 codes times s g, in fp32, rounded to the row's type.
template <typename T>
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t scale, float g) {
  const float z = __fmul_rn(e4m3_to_float(scale), g);
  uint32_t e[4], o[4];
  e2m1x8_to_half(codes, e);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 p = Elem<__half>::unpack(e[k]);
    o[k] = Elem<T>::pack(__fmul_rn(p.x, z), __fmul_rn(p.y, z));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) cache_fp4_read_kernel(const Fp4CacheArgs a) {
  grid_dependency_wait();  // the pool and the slots may come from the kernel before
  grid_launch_dependents();
  const int items = a.num_kv_heads * (D / 8);
  for_tokens<D>(a, gridDim.x, [&](int64_t token, int64_t slot, int item0) {
    uint4 *key = reinterpret_cast<uint4 *>(static_cast<T *>(a.key) + token * a.key_stride);
    uint4 *value = reinterpret_cast<uint4 *>(static_cast<T *>(a.value) + token * a.value_stride);
    const Place<D> at(a, slot, item0);
    const uint8_t *kc = static_cast<const uint8_t *>(a.k_cache) + at.tile0;
    const uint8_t *vc = static_cast<const uint8_t *>(a.v_cache) + at.tile0;
    for (int i0 = 0; item0 + i0 < items; i0 += 32 * kBatch) {
      uint32_t kq[kBatch], ks[kBatch], vq[kBatch], vs[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int off = (i0 / 32 + i) * at.step;
        if (item0 + i0 + 32 * i < items) {
          kq[i] = *reinterpret_cast<const uint32_t *>(kc + at.codes + off);
          vq[i] = *reinterpret_cast<const uint32_t *>(vc + at.codes + off);
          ks[i] = kc[at.scale + off];
          vs[i] = vc[at.scale + off];
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int item = item0 + i0 + 32 * i;
        if (item < items) {
          key[item] = values8<T>(kq[i], ks[i], a.k_scale);
          value[item] = values8<T>(vq[i], vs[i], a.v_scale);
        }
      }
    }
  });
}

// CTAs for the K and V rows of a call.
unsigned kv_ctas(int num_tokens, int num_kv_heads, int head_dim) {
  const int items = num_kv_heads * (head_dim / 8);
  const int per_cta = kWarps * (items < 32 ? 32 / items : 1);
  const int64_t ctas = (static_cast<int64_t>(num_tokens) + per_cta - 1) / per_cta;
  const int64_t most = kSms * PA_CACHE_FP4_CTAS;  // then a warp takes several tokens in turn
  return static_cast<unsigned>(ctas < most ? ctas : most);
}

template <typename K>
cudaError_t launch(K kern, const Fp4CacheArgs &a, cudaStream_t stream) {
  return launch_dependent(kern, dim3(kv_ctas(a.num_tokens, a.num_kv_heads, a.head_dim)),
                          dim3(kWarps * 32), 0, stream, a);
}

template <typename T, int D> cudaError_t launch_rope(RopeArgs a, cudaStream_t stream) {
  a.group_log2 = rope_group_log2(a.num_q_heads * (D / 16));
  const unsigned per_cta = kWarps * 32 >> a.group_log2;
  const unsigned kv = kv_ctas(a.num_tokens, a.num_kv_heads, D);
  return launch_dependent(cache_fp4_rope_kernel<T, D>,
                          dim3(kv + (a.num_tokens + per_cta - 1) / per_cta), dim3(kWarps * 32), 0,
                          stream, a, kv);
}

}  // namespace

cudaError_t launch_cache_fp4_write(const Fp4CacheArgs &a, int dtype, cudaStream_t stream) {
  if (dtype == 0)
    return a.head_dim == 128 ? launch(cache_fp4_write_kernel<__half, 128>, a, stream)
                             : launch(cache_fp4_write_kernel<__half, 64>, a, stream);
  return a.head_dim == 128 ? launch(cache_fp4_write_kernel<__nv_bfloat16, 128>, a, stream)
                           : launch(cache_fp4_write_kernel<__nv_bfloat16, 64>, a, stream);
}

cudaError_t launch_rope_fp4(const RopeArgs &a, int head_dim, int dtype, cudaStream_t stream) {
  if (dtype == 0)
    return head_dim == 128 ? launch_rope<__half, 128>(a, stream) : launch_rope<__half, 64>(a, stream);
  return head_dim == 128 ? launch_rope<__nv_bfloat16, 128>(a, stream)
                         : launch_rope<__nv_bfloat16, 64>(a, stream);
}

cudaError_t launch_cache_fp4_read(const Fp4CacheArgs &a, int dtype, cudaStream_t stream) {
  if (dtype == 0)
    return a.head_dim == 128 ? launch(cache_fp4_read_kernel<__half, 128>, a, stream)
                             : launch(cache_fp4_read_kernel<__half, 64>, a, stream);
  return a.head_dim == 128 ? launch(cache_fp4_read_kernel<__nv_bfloat16, 128>, a, stream)
                           : launch(cache_fp4_read_kernel<__nv_bfloat16, 64>, a, stream);
}

}  // namespace pa
